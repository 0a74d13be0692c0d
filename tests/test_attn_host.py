"""Attention operators on the host: refusals (every call fails before any CUDA call, so no
GPU is needed), the rotary table, and pins of the oracle."""
import ctypes

import numpy as np
import pytest
import torch

from gated_delta_rule_chunk_gb300 import binding as B
from gated_delta_rule_chunk_gb300.build import build
from gated_delta_rule_chunk_gb300.rope import rope_frequencies, rope_table
from oracle import attention as A


@pytest.fixture(scope="module")
def lib():
    build()
    return B.load_library()


def desc(**kw):
    base = dict(T=8, N=4, H=8, Hk=2, D=128, page_size=16, n_pages=9, max_pages=5, rot_dim=64,
                max_pos=80)
    base.update(kw)
    return B.make_attn_desc(**base)


@pytest.mark.parametrize("kw, want", [
    ({}, 0), (dict(D=64), 0), (dict(T=0), 0), (dict(page_size=0), 0), (dict(rot_dim=0), 0),
    (dict(page_size=256), 0), (dict(in_dtype=torch.float32), 0),
    (dict(T=-1), -2), (dict(N=0), -2), (dict(H=0), -2), (dict(Hk=0), -2), (dict(H=9), -2),
    (dict(n_pages=-1), -2), (dict(max_pages=-1), -2), (dict(rot_dim=-16), -2),
    (dict(rot_dim=144), -2), (dict(max_pos=-1), -2), (dict(page_size=-16), -2),
    (dict(max_pages=1 << 27), -2), (dict(T=1 << 30), -2),
    (dict(D=96), -3), (dict(D=256, rot_dim=0), -3), (dict(rot_dim=24), -3), (dict(page_size=48), -3),
    (dict(page_size=8), -3), (dict(page_size=512), -3), (dict(H=130, Hk=2), -3), (dict(flags=2), -3),
])
def test_check_desc(lib, kw, want):
    assert B.gdn_attn_check_desc(desc(**kw)) == want
    if want == 0 and desc(**kw).T:
        assert B.gdn_attn_workspace_size(desc(**kw)) > 0
    elif want:
        assert B.gdn_attn_workspace_size(desc(**kw)) == 0


def test_positions_stay_within_31_bits(lib):
    # a tile or copy that a sequence ends in reaches past its last position, before its clamp
    for page in (16, 32, 64, 128, 256):
        most = ((1 << 31) - 4096) // page
        assert B.gdn_attn_check_desc(desc(page_size=page, max_pages=most)) == 0
        assert B.gdn_attn_check_desc(desc(page_size=page, max_pages=most + 1)) == -2


def test_workspace_of_no_rows(lib):
    # a decode call without rows is allowed and asks for its workspace like any other
    for kw in (dict(T=0), dict(T=0, N=1, H=1, Hk=1, D=64), dict(T=0, N=300, H=64, Hk=64)):
        assert 0 < B.gdn_attn_workspace_size(desc(**kw)) <= B.gdn_attn_workspace_size(
            desc(**{**kw, "T": desc(**kw).N}))


def test_check_desc_null_and_dtype(lib):
    assert lib.gdn_attn_check_desc(None) == -1
    d = desc()
    d.in_dtype = 5
    assert B.gdn_attn_check_desc(d) == -3
    assert B.gdn_attn_workspace_size(desc(T=9)) == 0  # not a multiple of N


def call(fn, d, *args):
    conv = [ctypes.c_void_p(a) if type(a) is int else a for a in args]
    return fn(ctypes.byref(d), *conv)


FRONT = dict(x=16, qw=16, kw=16, rope=16, cu=16, kv=16, table=16, q=16, k=16, v=16, kc=16, vc=16)


@pytest.mark.parametrize("change, want", [
    (dict(x=None), -1), (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1),
    (dict(rope=None), -1), (dict(kc=None), -1), (dict(vc=None), -1), (dict(table=None), -1),
    (dict(cu=None), -2), (dict(x=24), -4), (dict(qw=8), -4), (dict(rope=20), -4), (dict(q=18), -4),
    (dict(kc=40), -4), (dict(cu=18), -4), (dict(kv=17), -4), (dict(table=19), -4),
])
def test_front_refuses(lib, change, want):
    a = {**FRONT, **change}
    assert call(lib.gdn_attn_front, desc(), *a.values(), None) == want


def test_front_refuses_by_desc(lib):
    assert call(lib.gdn_attn_front, desc(page_size=0), *FRONT.values(), None) == -2
    assert call(lib.gdn_attn_front, desc(max_pos=0), *FRONT.values(), None) == -2
    assert call(lib.gdn_attn_front, desc(D=32, rot_dim=0), *FRONT.values(), None) == -3
    assert lib.gdn_attn_front(None, *[ctypes.c_void_p(16)] * 12, None) == -1


@pytest.mark.parametrize("change, want", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(out=None), -1),
    (dict(cu=None), -2), (dict(q=8), -4), (dict(k=17), -4), (dict(v=24), -4), (dict(out=2), -4),
    (dict(cu=2), -4), (dict(lse=2), -4),
])
def test_prefill_refuses(lib, change, want):
    a = {**dict(q=16, k=16, v=16, cu=16, scale=0.0, out=16, lse=None), **change}
    a["scale"] = ctypes.c_float(0)
    assert call(lib.gdn_attn_prefill, desc(), *a.values(), None) == want


def test_prefill_refuses_f32(lib):
    p = ctypes.c_void_p(16)
    d = desc(in_dtype=torch.float32)
    assert lib.gdn_attn_prefill(ctypes.byref(d), p, p, p, p, 0.0, p, None, None) == -3


@pytest.mark.parametrize("change, kw, want", [
    (dict(q=None), {}, -1), (dict(kc=None), {}, -1), (dict(vc=None), {}, -1),
    (dict(table=None), {}, -1), (dict(kv=None), {}, -1), (dict(out=None), {}, -1),
    (dict(shared=8), {}, -2), (dict(shared=-16), {}, -2), (dict(shared=96), {}, -2),
    ({}, dict(T=9), -2), ({}, dict(page_size=0), -2), ({}, dict(T=4 * 17), -3),
    ({}, dict(in_dtype=torch.float32), -3),
    (dict(q=8), {}, -4), (dict(kc=8), {}, -4), (dict(vc=8), {}, -4), (dict(table=2), {}, -4),
    (dict(kv=2), {}, -4), (dict(out=8), {}, -4), (dict(lse=2), {}, -4),
])
def test_decode_refuses(lib, change, kw, want):
    a = {**dict(q=16, kc=16, vc=16, table=16, kv=16, shared=0, scale=0, out=16, lse=None), **change}
    d = desc(**kw)
    d.workspace = 4096
    d.workspace_bytes = 1 << 40
    f = lambda x: None if x is None else ctypes.c_void_p(x)
    assert lib.gdn_attn_decode(ctypes.byref(d), f(a["q"]), f(a["kc"]), f(a["vc"]), f(a["table"]),
                               f(a["kv"]), a["shared"], 0.0, f(a["out"]), f(a["lse"]), None) == want


def test_decode_refuses_workspace(lib):
    p = ctypes.c_void_p(16)
    d = desc()
    run = lambda: lib.gdn_attn_decode(ctypes.byref(d), p, p, p, p, p, 0, 0.0, p, None, None)
    assert run() == -1
    d.workspace = 4096
    d.workspace_bytes = B.gdn_attn_workspace_size(d) - 1
    assert run() == -5
    d.workspace = 4096 + 16
    d.workspace_bytes = 1 << 40
    assert run() == -4


def test_binding_refuses_cpu_tensors_and_shapes():
    x = torch.zeros(4, 6 * 128)
    with pytest.raises(ValueError):
        B.gdn_attn_front(x, 4, 1, 128)
    with pytest.raises(ValueError):
        B.gdn_attn_front(x, 4, 1, 128, cu_seqlens=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        B.gdn_attn_front(x.half(), 4, 1, 128)
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        B.gdn_attn_prefill(q, q, q)


def two_device_cases():
    """Each call with all its tensors on cuda:0 (stand-ins without memory: the refusal comes
    before anything is allocated, enqueued or looked at), and one of them on cuda:1."""
    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    front = dict(x=((8, 6 * 128), bf), q_weight=((128,), f32), k_weight=((128,), f32),
                 rope=((64, 32), f32), cu_seqlens=((3,), i32), kv_lens=((2,), i32),
                 page_table=((2, 4), i32), k_cache=((5, 1, 16, 128), bf),
                 v_cache=((5, 1, 16, 128), bf), q=((8, 4, 128), bf), k=((8, 1, 128), bf),
                 v=((8, 1, 128), bf), status=((1,), i32))
    prefill = dict(q=((8, 4, 128), bf), k=((8, 1, 128), bf), v=((8, 1, 128), bf),
                   cu_seqlens=((3,), i32), out=((8, 4, 128), bf), lse=((8, 4), f32),
                   status=((1,), i32))
    decode = dict(q=((2, 4, 128), bf), k_cache=((5, 1, 16, 128), bf), v_cache=((5, 1, 16, 128), bf),
                  page_table=((2, 4), i32), kv_lens=((2,), i32), out=((2, 4, 128), bf),
                  lse=((2, 4), f32), workspace=((1 << 24,), torch.uint8), status=((1,), i32))
    for call, shapes, rest in (("front", front, dict(H=4, Hk=1, D=128)), ("prefill", prefill, {}),
                               ("decode", decode, {})):
        for name in list(shapes)[1:]:
            yield pytest.param(call, shapes, rest, name, id=f"{call}-{name}")


@pytest.mark.parametrize("call, shapes, rest, away", list(two_device_cases()))
def test_binding_refuses_tensors_of_another_device(call, shapes, rest, away):
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        a = {n: torch.empty(shape, dtype=dtype, device="cuda:1" if n == away else "cuda:0")
             for n, (shape, dtype) in shapes.items()}
    with pytest.raises(ValueError, match=f"{away} is on cuda:1"):
        getattr(B, f"gdn_attn_{call}")(**a, **rest)


@pytest.mark.parametrize("call, flag", [("front", "interleaved"), ("front", "output_kv"),
                                        ("prefill", "return_lse"), ("decode", "return_lse")])
def test_flags_without_a_truth_value_are_errors(call, flag):
    """(stand-ins without memory: the error comes before anything is allocated or enqueued)"""
    from torch._subclasses.fake_tensor import FakeTensorMode

    class Neither:
        def __bool__(self):
            raise ZeroDivisionError
    with FakeTensorMode():
        x = torch.empty(8, 6 * 128, dtype=torch.bfloat16, device="cuda:0")
        q, k = (torch.empty(8, h, 128, dtype=torch.bfloat16, device="cuda:0") for h in (4, 1))
        kc = torch.empty(5, 1, 16, 128, dtype=torch.bfloat16, device="cuda:0")
        table, kv = (torch.empty(n, dtype=torch.int32, device="cuda:0") for n in ((8, 4), (8,)))
    args = dict(front=(x, 4, 1, 128), prefill=(q, k, k), decode=(q, kc, kc, table, kv))[call]
    with pytest.raises(ZeroDivisionError):
        getattr(B, f"gdn_attn_{call}")(*args, **{flag: Neither()})


@pytest.mark.parametrize("what", ["library", "module"])
def test_missing_builds_are_errors_at_once(what, lib, monkeypatch, tmp_path):
    import threading
    monkeypatch.setattr(B, "_lock", threading.Lock())
    monkeypatch.setattr(B, "_attn_module", None)
    monkeypatch.setattr(B, "_PKG", str(tmp_path))
    monkeypatch.setattr(B.build, "MODULE", str(tmp_path / "_attn_torch.so"))
    if what == "library":
        monkeypatch.setattr(B, "_lib", None)
    seen = []

    def call():
        try:
            B.load_library(str(tmp_path / "libgdn.so")) if what == "library" else B._attn()
        except B.GdnError as e:
            seen.append(str(e))
    t = threading.Thread(target=call, daemon=True)
    t.start()
    t.join(10)
    assert not t.is_alive() and len(seen) == 1 and "missing (build it" in seen[0]


# ---------------------------------------------------------------- the compiled marshalling
def test_module_of_another_torch_is_stale_and_refused(monkeypatch, lib):
    """The module is built against one torch and one Python: with others in their place it is
    built again, and until then not loaded."""
    from gated_delta_rule_chunk_gb300 import build as M
    assert M.module_up_to_date()
    monkeypatch.setattr(M, "module_abi", lambda: "another torch")
    assert not M.module_up_to_date()
    monkeypatch.setattr(B, "_attn_module", None)
    with pytest.raises(B.GdnError, match="build it"):
        B.gdn_attn_prefill(None, None, None)


@pytest.fixture
def small_build(monkeypatch, tmp_path):
    """build() of one small source into an empty folder."""
    from gated_delta_rule_chunk_gb300 import build as M
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(M, "_sources", lambda: [str(src)])
    for name, file in (("LIB", "libone.so"), ("BUILD", "_build"), ("MODULE", "_module.so"),
                       ("MODULE_STAMP", "_module.abi")):
        monkeypatch.setattr(M, name, str(tmp_path / file), raising=False)
    return M, tmp_path


def works(path):
    return ctypes.CDLL(str(path)).one() == 1


def test_library_is_built_without_torch(small_build, monkeypatch, capfd):
    import sys
    M, out = small_build
    monkeypatch.setitem(sys.modules, "torch", None)
    M.build()
    assert works(out / "libone.so") and not (out / "_module.so").exists()
    assert "torch" in capfd.readouterr().err
    M.build()  # and again, with the library up to date


def test_library_is_built_without_python_headers(small_build, monkeypatch, tmp_path):
    M, out = small_build
    monkeypatch.setattr(M.sysconfig, "get_paths", lambda: {"include": str(tmp_path / "none")})
    M.build()
    assert works(out / "libone.so") and not (out / "_module.so").exists()


def test_module_that_does_not_compile_leaves_the_library(small_build, monkeypatch):
    M, out = small_build
    bad = out / "bad.cpp"
    bad.write_text("#error no\n")
    monkeypatch.setattr(M, "MODULE_SRC", str(bad))
    with pytest.raises(RuntimeError, match="bad.cpp"):
        M.build()
    assert works(out / "libone.so") and not (out / "_module.so").exists()


# ---------------------------------------------------------------- rotary table
def test_rope_table_plain():
    t = rope_table(50, 8, base=100.0, device="cpu")
    assert t.shape == (50, 8) and t.dtype == torch.float32
    for p in (0, 1, 49):
        for i in range(4):
            a = p * 100.0 ** (-2 * i / 8)
            assert abs(t[p, i].item() - np.cos(a)) < 1e-7
            assert abs(t[p, 4 + i].item() - np.sin(a)) < 1e-7


def test_rope_scaling_rules():
    f = rope_frequencies(64)
    assert torch.allclose(rope_frequencies(64, linear=4.0), f / 4, rtol=1e-14)
    n = rope_frequencies(64, ntk=8.0)
    assert n[0] == f[0] and abs((f[-1] / n[-1]).item() - 8.0) < 1e-9
    b = rope_frequencies(64, by_parts=(8.0, 4096, 1.0, 32.0))
    turns = f * 4096 / (2 * np.pi)
    assert torch.equal(b[turns > 32], f[turns > 32])
    assert torch.allclose(b[turns < 1], f[turns < 1] / 8, rtol=1e-14)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and ((b[mid] > f[mid] / 8) & (b[mid] < f[mid])).all()
    assert torch.equal(rope_table(9, 16, magnitude=1.5, device="cpu")[0, :8], torch.full((8,), 1.5))
    with pytest.raises(ValueError):
        rope_frequencies(7)
    with pytest.raises(ValueError):
        rope_frequencies(8, by_parts=(8.0, 4096, 2.0, 2.0))


# ---------------------------------------------------------------- oracle pins
def test_oracle_attention_closed_forms():
    rng = np.random.default_rng(0)
    v = rng.normal(size=(7, 4))
    q = np.zeros((7, 4))  # equal scores: running means
    out, _, lse = A.attend(q, rng.normal(size=(7, 4)), v, np.arange(7), 1.0)
    np.testing.assert_allclose(out, np.cumsum(v, 0) / np.arange(1, 8)[:, None], rtol=1e-12)
    np.testing.assert_allclose(lse, np.log(np.arange(1, 8)), rtol=1e-12)
    k = np.eye(4) * 1e4  # one key takes all
    out, _, _ = A.attend(np.eye(4), k, v[:4], np.full(4, 3), 1.0)
    np.testing.assert_allclose(out, v[:4], rtol=1e-12)
    out, _, lse = A.attend(q, k, v[:4], np.full(7, -1), 1.0)  # nothing seen
    assert not out.any() and np.isneginf(lse).all()


def test_oracle_decode_equals_prefill_last_row():
    rng = np.random.default_rng(1)
    L, H, Hk, D, page = 37, 4, 2, 8, 16
    q, k, v = (rng.normal(size=(L, h, D)) for h in (H, Hk, Hk))
    out, _, lse, _ = A.prefill(q, k, v)
    table = np.array([[2, 0, 1]])
    kc, vc = np.full((3, Hk, page, D), np.nan), np.full((3, Hk, page, D), np.nan)
    for t in range(L):
        kc[table[0, t // page], :, t % page], vc[table[0, t // page], :, t % page] = k[t], v[t]
    for shared in (0, 16, 32):
        o, _, l = A.decode(q[None, -3:], kc, vc, table, [L], shared)
        np.testing.assert_allclose(o[0], out[-3:], rtol=1e-12)
        np.testing.assert_allclose(l[0], lse[-3:], rtol=1e-12)


def test_oracle_front_rotation_keeps_relative_position():
    """q . k after rotation depends on the distance only, and each pair's norm is kept."""
    rng = np.random.default_rng(2)
    D, rot = 16, 8
    x = rng.normal(size=(1, 3 * D))
    for inter in (False, True):
        table = rope_table(40, rot, base=50.0, device="cpu").double().numpy()
        dots = []
        for p in (3, 30):
            q = A.front(x, 1, 1, D, rope=table, interleaved=inter, kv_lens=[p + 1])[0][0, 0]
            k = A.front(x, 1, 1, D, rope=table, interleaved=inter, kv_lens=[p - 2])[1][0, 0]
            dots.append(q @ k)
            np.testing.assert_allclose(np.linalg.norm(q), np.linalg.norm(x[0, :D]), rtol=1e-6)
        np.testing.assert_allclose(dots[0], dots[1], rtol=1e-5)
