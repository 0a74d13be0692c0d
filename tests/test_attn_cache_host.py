"""Long-conversation operators without a GPU: the oracle's pins, and what the calls refuse."""
import ctypes

import numpy as np
import pytest
import torch

from gated_delta_rule_chunk_gb300 import binding as B
from oracle import attention as A
from oracle import attention_cache as C


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g
    g.build()
    return B.load_library()


# ---------------------------------------------------------------- oracle
def test_e4m3_values_are_torchs():
    b = torch.arange(256, dtype=torch.uint8)
    want = b.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.nan_to_num(C.VALUES, nan=-1e9), np.nan_to_num(want, nan=-1e9))


def test_e4m3_rounding_is_to_nearest_even():
    g = torch.Generator().manual_seed(0)
    x = torch.cat([torch.randn(20000, generator=g) * 10.0 ** e for e in (-3, -2, 0, 1)]).clamp(-448, 448)
    mids = torch.from_numpy((C.VALUES[:126] + C.VALUES[1:127]) / 2).float()
    x = torch.cat([x, mids, -mids, torch.tensor([0.0, 448.0, -448.0, 2.0 ** -10, 2.0 ** -9])])
    want = x.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert C.same_bytes(C.to_e4m3(x.double().numpy()), want).all()


def test_scale_fits_and_is_the_least():
    for top in (448.0, 448.0 * 2 ** 0.01, 1.0, 3.5, 3.6, 1e-20, 1e30, 2.0 ** -126):
        s = C.least_scale(top)
        assert top <= 448 * s and (top > 224 * s or s == 2.0 ** -100)
    assert C.least_scale(0.0) == 2.0 ** -100


def test_append_in_parts_holds_the_same_where_the_scale_does_not_grow():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((40, 2, 64)) * 2.0 ** rng.integers(-3, 4, (40, 1, 1))
    x[::16] = 100.0 * x[::16]  # each block's largest token first
    table = np.array([[2, 0, 1]])
    cache, scale = np.zeros((3, 2, 16, 64), np.uint8), np.zeros((3, 2, 1), np.float32)
    one = C.append8(x, cache, scale, table)
    for at in range(40):
        cache, scale = C.append8(x[at:at + 1], cache, scale, table, [at + 1])
    assert np.array_equal(one[0], cache) and np.array_equal(one[1], scale)


def test_a_value_is_held_to_its_rounding():
    """Half a step of e4m3 (2^-4 of the value), or of its least step times the scale."""
    rng = np.random.default_rng(2)
    x = rng.standard_normal((16, 1, 64)) * 10.0 ** rng.uniform(-3, 3, (16, 1, 64))
    cache, scale = C.append8(x, np.zeros((1, 1, 16, 64), np.uint8), np.zeros((1, 1, 1)), np.array([[0]]))
    got = C.held(cache, scale)[0].transpose(1, 0, 2)
    assert (np.abs(got - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * scale.max())).all()


def test_decode_weights_of_one_row_sum_to_one():
    rng = np.random.default_rng(3)
    q, k = rng.standard_normal((1, 1, 2, 64)), rng.standard_normal((3, 1, 16, 64))
    w = C.decode_weights(q, k, np.array([[1, 2]]), [20], np.zeros((3, 1, 16)))
    assert abs(w.sum() - 2) < 1e-12 and (w[0] == 0).all() and (w[2, 0, 4:] == 0).all()


def test_prompt_weights_are_those_of_its_decode_steps():
    rng = np.random.default_rng(4)
    L, table = 23, np.array([[1, 0]])
    q, k = rng.standard_normal((L, 2, 64)), rng.standard_normal((L, 1, 64))
    lse = A.prefill(q, k, k)[2]
    want = np.zeros((2, 1, 16))
    cache = np.zeros((2, 1, 16, 64))
    for t in range(L):
        cache[table[0, t // 16], 0, t % 16] = k[t, 0]
        want = C.decode_weights(q[None, t:t + 1], cache, table, [t + 1], want)
    got = C.prefill_weights(q, k, lse, np.zeros((2, 1, 16)), table)
    assert np.abs(got - want).max() < 1e-12
    last = C.prefill_weights(q, k, lse, np.zeros((2, 1, 16)), table, window=1)
    assert abs(last.sum() - 2) < 1e-12


def test_choice():
    w = np.array([1.0, 5.0, 5.0, 0.0, -0.0, 2.0, 9.0])
    assert C.choose(w, 7, 1) == list(range(7))
    assert C.choose(w, 3, 1) == [1, 2, 6]
    assert C.choose(w, 2, 0) == [1, 6]
    assert C.choose(w, 2, 2) == [5, 6]
    assert C.choose(np.array([0.0, -0.0, 0.0, 1.0]), 2, 1) == [0, 3]
    assert C.choose(np.array([np.inf, np.nan, 3.0, 1.0]), 2, 1) == [1, 3]


def test_axes_all_alike_are_the_plain_positions():
    rng = np.random.default_rng(5)
    T, H, Hk, D = 7, 2, 1, 64
    x, rope = rng.standard_normal((T, 4 * D)), rng.standard_normal((20, 32))
    pos = np.arange(T)[None] + 3
    a = C.front_axes(x, H, Hk, D, None, None, 1e-6, rope, False, np.repeat(pos, 3, 0), np.arange(16) % 3)
    b = A.front(x, H, Hk, D, rope=rope, kv_lens=[T + 3], cu=[0, T])
    assert np.allclose(a[0], b[0]) and np.allclose(a[1], b[1])


# ---------------------------------------------------------------- refusals of the C ABI
def desc(**kw):
    a = dict(T=8, N=2, H=4, Hk=1, D=128, page_size=16, n_pages=6, max_pages=4, rot_dim=32, max_pos=64)
    return B.make_attn_desc(**{**a, **kw})


def ptr(x):
    return None if x is None else ctypes.c_void_p(x)


AXES = dict(x=16, qw=16, kw=16, rope=16, cu=16, kv=16, pos=16, n_axes=3, axes=16, table=16, q=16, k=16,
            v=16, kc=16, vc=16)


@pytest.mark.parametrize("change, kw, want", [
    (dict(pos=None), {}, -1), (dict(n_axes=0), {}, -2), (dict(n_axes=9), {}, -2),
    ({}, dict(rot_dim=0), -2), (dict(pos=18), {}, -4), (dict(axes=17), {}, -4), (dict(x=None), {}, -1),
    (dict(rope=None), {}, -1), (dict(kc=None), {}, -1), ({}, dict(max_pos=0), -2), ({}, dict(D=96), -3),
])
def test_front_axes_refuses(lib, change, kw, want):
    a = {n: x if n == "n_axes" else ptr(x) for n, x in {**AXES, **change}.items()}
    assert lib.gdn_attn_front_axes(ctypes.byref(desc(**kw)), *a.values(), None) == want


APPEND = dict(k=16, v=16, cu=16, kv=16, table=16, kc=16, vc=16, ks=16, vs=16)


@pytest.mark.parametrize("change, kw, want", [
    *[({n: None}, {}, -1) for n in APPEND if n not in ("cu", "kv")], (dict(cu=None), {}, -2),
    ({}, dict(page_size=0), -2), ({}, dict(page_size=24), -3), ({}, dict(D=32, rot_dim=0), -3),
    (dict(k=24), {}, -4), (dict(v=8), {}, -4), (dict(kc=8), {}, -4), (dict(vc=24), {}, -4),
    (dict(ks=2), {}, -4), (dict(vs=18), {}, -4), (dict(table=17), {}, -4), (dict(kv=18), {}, -4),
])
def test_append8_refuses(lib, change, kw, want):
    a = [ptr(x) for x in {**APPEND, **change}.values()]
    assert lib.gdn_attn_append8(ctypes.byref(desc(**kw)), *a, None) == want


DECODE = dict(q=16, kc=16, vc=16, ks=16, vs=16, table=16, kv=16, shared=0, scale=0.0, out=16, lse=None,
              weights=None)


@pytest.mark.parametrize("change, kw, want", [
    (dict(q=None), {}, -1), (dict(kc=None), {}, -1), (dict(ks=None), {}, -1), (dict(vs=None), {}, -1),
    (dict(kv=None), {}, -1), (dict(out=None), {}, -1), (dict(shared=8), {}, -2), (dict(shared=96), {}, -2),
    (dict(weights=16, shared=16), {}, -3), (dict(weights=18), {}, -4), (dict(ks=18), {}, -4),
    (dict(vs=17), {}, -4), (dict(lse=2), {}, -4), (dict(kc=8), {}, -4), ({}, dict(T=9), -2),
    ({}, dict(T=4 * 17), -3), ({}, dict(in_dtype=torch.float32), -3), ({}, dict(page_size=0), -2),
])
def test_decode_cache_refuses(lib, change, kw, want):
    a = {n: x if n in ("shared", "scale") else ptr(x) for n, x in {**DECODE, **change}.items()}
    d = desc(**kw)
    d.workspace = 4096
    d.workspace_bytes = 1 << 40
    assert lib.gdn_attn_decode_cache(ctypes.byref(d), *a.values(), None) == want


@pytest.mark.parametrize("weights", [False, True])
def test_decode_cache_refuses_workspace(lib, weights):
    a = {n: x if n in ("shared", "scale") else ptr(x)
         for n, x in {**DECODE, "weights": 16 if weights else None}.items()}
    d = desc()
    run = lambda: lib.gdn_attn_decode_cache(ctypes.byref(d), *a.values(), None)
    assert run() == -1
    d.workspace = 4096
    d.workspace_bytes = B.gdn_attn_decode_cache_workspace_size(d, weights) - 1
    assert run() == -5
    d.workspace, d.workspace_bytes = 4096 + 64, 1 << 40
    assert run() == -4
    assert B.gdn_attn_decode_cache_workspace_size(desc(T=9), weights) == 0


PROMPT = dict(q=16, k=16, lse=16, cu=16, table=16, window=0, scale=0.0, weights=16)


@pytest.mark.parametrize("change, kw, want", [
    *[({n: None}, {}, -1) for n in ("q", "k", "lse", "table", "weights")], (dict(cu=None), {}, -2),
    (dict(window=-1), {}, -2), ({}, dict(page_size=0), -2), ({}, dict(in_dtype=torch.float32), -3),
    (dict(q=8), {}, -4), (dict(k=24), {}, -4), (dict(lse=18), {}, -4), (dict(weights=17), {}, -4),
    (dict(scale=2.0 ** -101), {}, -3), (dict(scale=1e-45), {}, -3),
])
def test_prefill_weights_refuses(lib, change, kw, want):
    a = {n: x if n in ("window", "scale") else ptr(x) for n, x in {**PROMPT, **change}.items()}
    d = desc(**kw)
    run = lambda: lib.gdn_attn_prefill_weights(ctypes.byref(d), *a.values(), None)
    d.workspace, d.workspace_bytes = 4096, 1 << 40
    assert run() == want
    if not change and not kw:
        return
    d = desc()
    a = {n: x if n in ("window", "scale") else ptr(x) for n, x in PROMPT.items()}
    assert run() == -1
    d.workspace, d.workspace_bytes = 4096, B.gdn_attn_prefill_weights_workspace_size(d) - 1
    assert run() == -5


EVICT = dict(kc=16, vc=16, ks=16, vs=16, weights=16, table=16, kv=16, new=16, new_max=2, keep=20, recent=3,
             lens=16, kept=16)


@pytest.mark.parametrize("change, kw, want", [
    *[({n: None}, {}, -1) for n in EVICT if n not in ("new_max", "keep", "recent")],
    (dict(keep=0), {}, -2), (dict(keep=33), {}, -2), (dict(recent=21), {}, -2), (dict(recent=-1), {}, -2),
    (dict(new_max=0), {}, -2), ({}, dict(page_size=0), -2), ({}, dict(D=32, rot_dim=0), -3),
    (dict(kc=8), {}, -4), (dict(vc=24), {}, -4), (dict(ks=18), {}, -4), (dict(weights=17), {}, -4),
    (dict(new=18), {}, -4), (dict(lens=18), {}, -4), (dict(kept=17), {}, -4), (dict(kv=17), {}, -4),
])
def test_evict_refuses(lib, change, kw, want):
    a = {n: x if n in ("new_max", "keep", "recent") else ptr(x) for n, x in {**EVICT, **change}.items()}
    assert lib.gdn_attn_evict(ctypes.byref(desc(**kw)), *a.values(), None) == want


# ---------------------------------------------------------------- refusals of the binding
def cases():
    """Each call with tensors on cuda:0 without memory (the refusal comes before anything is
    allocated, enqueued or looked at)."""
    bf, i32, f32, f8 = torch.bfloat16, torch.int32, torch.float32, torch.float8_e4m3fn
    cache = dict(k_cache=((5, 1, 32, 128), f8), v_cache=((5, 1, 32, 128), f8),
                 k_scale=((5, 1, 2), f32), v_scale=((5, 1, 2), f32))
    front = dict(x=((8, 6 * 128), bf), rope=((64, 32), f32), positions=((3, 8), i32),
                 rope_axes=((16,), torch.uint8))
    append = dict(k=((8, 1, 128), bf), v=((8, 1, 128), bf), **cache, page_table=((2, 4), i32),
                  kv_lens=((2,), i32), cu_seqlens=((3,), i32), status=((1,), i32))
    decode = dict(q=((2, 4, 128), bf), **cache, page_table=((2, 4), i32), kv_lens=((2,), i32),
                  weights=((5, 1, 32), f32))
    prompt = dict(q=((8, 4, 128), bf), k=((8, 1, 128), bf), lse=((8, 4), f32), weights=((5, 1, 32), f32),
                  page_table=((2, 4), i32), cu_seqlens=((3,), i32), workspace=((1 << 24,), torch.uint8),
                  status=((1,), i32))
    evict = dict(**cache, weights=((5, 1, 32), f32), page_table=((2, 4), i32), kv_lens=((2,), i32),
                 new_table=((2, 1), i32), new_lens=((2,), i32), kept=((2, 1, 20), i32), status=((1,), i32))
    return dict(front=(front, dict(H=4, Hk=1, D=128)), append8=(append, {}), decode=(decode, {}),
                prefill_weights=(prompt, {}), evict=(evict, dict(keep=20)))


def tensors(shapes, change=None):
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        return {n: torch.empty(s, dtype=t, device="cuda:0") if n != change else None
                for n, (s, t) in shapes.items()}


@pytest.mark.parametrize("call, away", [(c, n) for c, (s, _) in cases().items() for n in list(s)
                                        if n not in ("x", "q") and (c, n) not in (
                                            ("append8", "k"), ("evict", "k_cache"))])
def test_binding_refuses_tensors_of_another_device(call, away):
    from torch._subclasses.fake_tensor import FakeTensorMode
    shapes, rest = cases()[call]
    a = tensors(shapes)
    with FakeTensorMode():
        a[away] = torch.empty(shapes[away][0], dtype=shapes[away][1], device="cuda:1")
    with pytest.raises(ValueError, match=f"{away} is on cuda:1"):
        getattr(B, f"gdn_attn_{call}")(**a, **rest)


@pytest.mark.parametrize("call, name, shape, dtype", [
    ("front", "positions", (3, 7), None), ("front", "positions", (24,), None),
    ("front", "rope_axes", (15,), None), ("front", "rope_axes", None, torch.int32),
    ("append8", "v", (8, 2, 128), None), ("append8", "k_cache", None, torch.bfloat16),
    ("append8", "k_scale", (5, 1, 32), None), ("append8", "v_scale", None, torch.bfloat16),
    ("append8", "kv_lens", (3,), None), ("append8", "k", None, torch.float16),
    ("decode", "k_cache", None, torch.bfloat16), ("decode", "k_scale", (5, 1, 1), None),
    ("decode", "weights", (5, 32), None), ("decode", "weights", None, torch.float64),
    ("prefill_weights", "lse", (4, 8), None), ("prefill_weights", "weights", (5, 2, 32), None),
    ("prefill_weights", "k", (9, 1, 128), None), ("prefill_weights", "lse", None, torch.bfloat16),
    ("evict", "weights", (5, 1, 16), None), ("evict", "kept", (2, 1, 21), None),
    ("evict", "v_scale", (5, 2), None), ("evict", "v_cache", None, torch.uint8),
    ("evict", "new_table", (3, 1), None), ("evict", "new_lens", (3,), None),
])
def test_binding_refuses_shapes_and_types(call, name, shape, dtype):
    shapes, rest = cases()[call]
    s, t = shapes[name]
    with pytest.raises((ValueError, TypeError), match=f"{name}|unsupported dtype"):
        getattr(B, f"gdn_attn_{call}")(**refused(shapes, {name: (shape or s, dtype or t)}), **rest)


def refused(shapes, change):
    """CPU-only stand-ins that look like CUDA tensors up to the refusal; outputs given, so that
    nothing is allocated."""
    full = {**shapes, **change}
    if "x" in full:
        full.update(q=((8, 4, 128), torch.bfloat16), k=((8, 1, 128), torch.bfloat16),
                    v=((8, 1, 128), torch.bfloat16))
    if "k_cache" in full and "q" in full:
        full.update(out=((2, 4, 128), torch.bfloat16), workspace=((1 << 24,), torch.uint8))
    return tensors(full)


@pytest.mark.parametrize("call, missing", [("decode", "v_scale"), ("decode", "k_scale"),
                                           ("evict", "v_scale"), ("append8", "k_scale"),
                                           ("prefill_weights", "lse"), ("evict", "new_table")])
def test_binding_refuses_half_a_set(call, missing):
    shapes, rest = cases()[call]
    a = refused(shapes, {})
    a[missing] = None
    with pytest.raises((TypeError, B.GdnError, ValueError)):
        getattr(B, f"gdn_attn_{call}")(**a, **rest)


def test_binding_refuses_other_arguments():
    shapes, rest = cases()["front"]
    a = refused(shapes, {})
    with pytest.raises(ValueError, match="rope_axes needs positions"):
        B.gdn_attn_front(**{**a, "positions": None}, **rest)
    with pytest.raises(ValueError, match="need rope"):
        B.gdn_attn_front(**{**a, "rope": None}, **rest)
    shapes, rest = cases()["evict"]
    with pytest.raises(ValueError, match="keep"):
        B.gdn_attn_evict(**tensors(shapes), keep=0)


@pytest.mark.parametrize("change, error, text", [
    (dict(keep=33), B.GdnError, "gdn_attn_evict"), (dict(keep=1 << 30), B.GdnError, "gdn_attn_evict"),
    (dict(keep=1 << 40), ValueError, "32 bits"), (dict(recent=21), B.GdnError, "gdn_attn_evict"),
    (dict(recent=-1), B.GdnError, "gdn_attn_evict"),
])
def test_evict_refuses_a_budget_before_it_allocates(lib, change, error, text):
    """`kept` goes by the budget: one that the new pages do not hold is refused, not asked for."""
    shapes, _ = cases()["evict"]
    given = {n: x for n, x in shapes.items() if n not in ("new_lens", "kept")}
    with pytest.raises(error, match=text):
        B.gdn_attn_evict(**tensors(given), **{**dict(keep=20), **change})


def test_decode_refuses_weights_behind_a_prefix_before_it_allocates(lib):
    """The workspace holds the scores of all keys: not asked for by a call that is refused."""
    shapes, _ = cases()["decode"]
    a = tensors({n: x for n, x in shapes.items() if n not in ("k_scale", "v_scale")} |
                {n: (shapes[n][0], torch.bfloat16) for n in ("k_cache", "v_cache")})
    with pytest.raises(B.GdnError, match="gdn_attn_decode"):
        B.gdn_attn_decode(**a, shared_len=32)
    with pytest.raises(B.GdnError, match="gdn_attn_decode"):
        B.gdn_attn_decode(**tensors(shapes), shared_len=32)
