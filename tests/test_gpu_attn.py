"""Attention operators through the C ABI against the fp64 oracle.

Tolerances, derived before the first run:
  - attention, fp32 output: each weight may be rounded to bf16 (relative 2^-8 at most), which
    moves an output by at most 2^-8 sum_j w_ij |v_j|; scores (fp32 sums of D exact products)
    and exp add less than 2^-11 of the same sum at these inputs. A bf16 output adds half a
    unit in its last place, 2^-8 |o|. For one key the weight is 1 and exact.
  - lse: fp32 throughout; D roundings of partial sums of q . k, at most 2^-24 * D * sum |q k|,
    scaled; 1e-3 covers the largest score used here (sum |q k| scale < 600).
  - front: fp32 arithmetic of about ten roundings, 2e-6 relative to the pair's size (a
    rotation mixes both); a bf16 result adds 2^-8 of its own size.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_chunk_gb300 import binding as B
from gated_delta_rule_chunk_gb300.rope import rope_table
from oracle import attention as A

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
REL = 2.0 ** -8 + 2.0 ** -11


def randn(g, *shape, dtype=BF, mul=1.0):
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * mul).to(dtype)


def np64(x):
    return x.detach().double().cpu().numpy()


def close_attention(out, lse, ref, mag, ref_lse, rows=None):
    o = np64(out).reshape(ref.shape)
    rows = np.ones(ref.shape[0], bool) if rows is None else rows
    tol = REL * mag + (2.0 ** -8 * np.abs(ref) if out.dtype == BF else 0.0) + 1e-6
    bad = ~(np.abs(o - ref) <= tol)
    bad[~rows] = False
    assert not bad.any(), (np.argwhere(bad)[:5], o[bad][:5], ref[bad][:5], tol[bad][:5])
    if lse is not None:
        got = np64(lse).reshape(ref_lse.shape)[rows]
        want = ref_lse[rows]
        assert np.array_equal(np.isneginf(got), np.isneginf(want))
        fin = np.isfinite(want)
        assert np.abs(got[fin] - want[fin]).max(initial=0.0) <= 1e-3


# ---------------------------------------------------------------- prefill
@pytest.fixture(params=["by rule", "two"])
def row_tiles(request):
    """Work items of one or two row tiles as the sizes have it (one, in small tests), and of
    two always."""
    B.gdn_test_attn_tiles(2 if request.param == "two" else 0)
    yield
    B.gdn_test_attn_tiles(0)


either = pytest.mark.usefixtures("row_tiles")


def run_prefill(lens, H, Hk, D, seed=0, lead=0, tail=0, mul=1.0, scale=None, out_dtype=F32,
                spoil=None):
    g = torch.Generator().manual_seed(seed)
    T = lead + sum(lens) + tail
    q, k, v = randn(g, T, H, D, mul=mul), randn(g, T, Hk, D, mul=mul), randn(g, T, Hk, D)
    if spoil:
        spoil(q, k, v)
    cu = torch.tensor([lead] + lens).cumsum(0).to(torch.int32)
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    out = torch.full((T, H, D), 7.0, dtype=out_dtype, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    B.gdn_attn_prefill(q.cuda(), k.cuda(), v.cuda(), cu.cuda(), scale=scale, out=out, return_lse=True,
                       lse=lse, status=status)
    assert status.item() == 0
    return q, k, v, cu, out, lse


def check_prefill(*a, **kw):
    q, k, v, cu, out, lse = run_prefill(*a, **kw)
    ref, mag, rl, inside = A.prefill(np64(q), np64(k), np64(v), cu.numpy(), kw.get("scale"))
    close_attention(out, lse, ref, mag, rl, inside)
    assert (out[torch.tensor(~inside)] == 7.0).all() and (lse[torch.tensor(~inside)] == 7.0).all()


@either
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("L", [1, 2, 31, 63, 64, 65, 127, 128, 129, 255, 257, 400])
def test_prefill_lengths(L, D):
    check_prefill([L], 2, 1, D, seed=L)


@either
@pytest.mark.parametrize("H, Hk", [(1, 1), (3, 3), (3, 1), (5, 1), (6, 2), (7, 1), (8, 1), (16, 2),
                                   (24, 2), (33, 1), (64, 1)])
def test_prefill_groups(H, Hk):
    check_prefill([70, 1, 150], H, Hk, 128, seed=H)


@either
@pytest.mark.parametrize("lens", [[0, 5, 0, 130, 1, 0], [300, 1, 1, 64], [128, 128], [1] * 70,
                                  [3, 250, 17, 129, 66]])
@pytest.mark.parametrize("D", [64, 128])
def test_prefill_packed(lens, D):
    check_prefill(lens, 4, 2, D, seed=len(lens), lead=3, tail=9)


@either
def test_prefill_many_sequences():
    """More sequences than one launch takes, empty ones among them."""
    check_prefill([1 + 13 * i % 9 if i % 5 else 0 for i in range(1100)] + [140, 0, 3], 2, 1, 64, seed=7)


@either
@pytest.mark.parametrize("mul", [0.01, 4.0, 8.0])
def test_prefill_score_ranges(mul):
    """Nearly uniform weights, and weights of a few keys whose maximum grows along the row."""
    check_prefill([385], 2, 1, 128, mul=mul, seed=3, out_dtype=F32)


@either
def test_prefill_growing_maximum():
    """Every block of keys scores far above the one before: each running maximum is replaced."""
    def spoil(q, k, v):
        q[:] = 1.0
        k[:] = (torch.arange(k.shape[0]) / 8).floor()[:, None, None].to(k.dtype) / 16
    check_prefill([500], 2, 1, 128, spoil=spoil)

    def falling(q, k, v):
        q[:] = 1.0
        k[:] = (-(torch.arange(k.shape[0]) / 8).floor())[:, None, None].to(k.dtype) / 16
    check_prefill([500], 2, 1, 64, spoil=falling)


@either
def test_prefill_scale_and_bf16_output():
    check_prefill([200], 4, 1, 128, scale=0.3, seed=5)
    check_prefill([200], 4, 1, 64, seed=6, out_dtype=BF)


@either
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("what", ["nan", "inf", "lowest"])
def test_prefill_unseen_values_have_no_influence(what, D):
    """Keys and values from row 130 on, and the rows around the sequences, hold NaN, infinities
    or the type's lowest value: rows before 130 come out as if they held zeros."""
    bad = dict(nan=float("nan"), inf=float("inf"), lowest=torch.finfo(BF).min)[what]

    def spoil(q, k, v):
        for x in (k, v):
            x[:2] = bad
            x[2 + 130:2 + 200] = bad
            x[-5:] = bad
    lens = [200, 90]
    q, k, v, cu, out, lse = run_prefill(lens, 4, 2, D, lead=2, tail=5, spoil=spoil)
    kz, vz = np64(k), np64(v)
    for x in (kz, vz):
        x[2 + 130:2 + 200] = 0
    ref, mag, rl, inside = A.prefill(np64(q), kz, vz, cu.numpy())
    inside[2 + 130:2 + 200] = False
    close_attention(out, lse, ref, mag, rl, inside)
    if what == "nan":
        assert torch.isnan(out[2 + 130:2 + 200]).all()  # NaN that is seen is not hidden


@either
def test_prefill_one_nan_value_reaches_only_the_rows_that_see_it():
    def spoil(q, k, v):
        v[77, 0, 5] = float("nan")
    q, k, v, cu, out, lse = run_prefill([190], 2, 1, 128, spoil=spoil)
    vz = np64(v)
    vz[77, 0, 5] = 0
    ref, mag, rl, _ = A.prefill(np64(q), np64(k), vz)
    assert torch.isnan(out[77:, :, 5]).all()
    keep = torch.ones(128, dtype=torch.bool)
    keep[5] = False
    close_attention(out[..., keep], lse, ref[..., keep.numpy()], mag[..., keep.numpy()], rl)
    close_attention(out[:77], lse[:77], ref[:77], mag[:77], rl[:77])


def same_where_not_finite(out, ref):
    """NaN and infinities where the formula has them, with their signs."""
    o = np64(out).reshape(ref.shape)
    assert np.array_equal(np.isnan(o), np.isnan(ref))
    assert np.array_equal(np.isposinf(o), np.isposinf(ref))
    assert np.array_equal(np.isneginf(o), np.isneginf(ref))


@either
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_prefill_infinities_where_they_are_seen(D, out_dtype):
    """Values that are not finite at keys in and outside tiles with masked keys, several in one
    column: each row has of them what it sees."""
    inf, nan = float("inf"), float("nan")
    spots = [(0, 0, 3, inf), (70, 1, 5, -inf), (129, 0, 3, inf), (130, 0, 7, -inf), (131, 0, 7, inf),
             (200, 1, D - 1, nan), (255, 0, 0, inf), (256, 1, 9, -inf), (299, 0, 11, nan),
             (300, 0, 1, inf), (340, 1, D // 2, -inf), (379, 1, 2, inf)]  # the second prompt: 300 on

    def spoil(q, k, v):
        for t, h, d, x in spots:
            v[t, h, d] = x

    q, k, v, cu, out, lse = run_prefill([300, 80], 4, 2, D, seed=21, out_dtype=out_dtype, spoil=spoil)
    with np.errstate(invalid="ignore"):
        ref, mag, rl, inside = A.prefill(np64(q), np64(k), np64(v), cu.numpy(), None)
    same_where_not_finite(out, ref)
    o, fin = np64(out).reshape(ref.shape), np.isfinite(ref)
    tol = REL * mag[fin] + (2.0 ** -8 * np.abs(ref[fin]) if out_dtype == BF else 0.0) + 1e-6
    assert (np.abs(o[fin] - ref[fin]) <= tol).all() and fin.mean() > 0.5
    assert np.abs(np64(lse) - rl.reshape(lse.shape)).max() <= 1e-3


@either
def test_prefill_malformed_cu_seqlens():
    g = torch.Generator().manual_seed(1)
    q, k, v = (randn(g, 300, h, 64).cuda() for h in (4, 2, 2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for cu in ([0, 200, 100, 260], [-5, 90, 999], [50, 40, 30, 290], [7, 400, 20]):
        sane = torch.tensor(A.sane_bounds(cu, 300), dtype=torch.int32).cuda()
        outs = []
        for c in (torch.tensor(cu, dtype=torch.int32).cuda(), sane):
            out = torch.zeros(300, 4, 64, dtype=BF, device="cuda")
            B.gdn_attn_prefill(q, k, v, c, out=out, status=status)
            outs.append((out, status.item()))
        assert outs[0][1] == 1 and outs[1][1] == 0
        assert torch.equal(outs[0][0], outs[1][0])


@either
def test_prefill_repeatable_other_stream_and_graph():
    g = torch.Generator().manual_seed(2)
    q, k, v = (randn(g, 700, h, 128).cuda() for h in (8, 2, 2))
    cu = torch.tensor([0, 333, 700], dtype=torch.int32).cuda()
    a = B.gdn_attn_prefill(q, k, v, cu)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = torch.empty_like(a)
    B.gdn_attn_prefill(q, k, v, cu, out=b, stream=s)
    s.synchronize()
    assert torch.equal(a, b)
    c = torch.zeros_like(a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.gdn_attn_prefill(q, k, v, cu, out=c)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, c)
    cu.copy_(torch.tensor([0, 100, 650], dtype=torch.int32))  # other lengths, same graph
    graph.replay()
    d = B.gdn_attn_prefill(q, k, v, cu, out=a.clone())
    torch.cuda.synchronize()
    assert torch.equal(c[:650], d[:650])


@pytest.mark.parametrize("lens, H, Hk, D", [([700, 3, 129, 64], 6, 2, 128), ([900, 130], 4, 4, 64)])
def test_prefill_same_with_one_or_two_tiles(lens, H, Hk, D):
    g = torch.Generator().manual_seed(12)
    q, k, v = (randn(g, sum(lens), h, D).cuda() for h in (H, Hk, Hk))
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).cuda()
    res = []
    for tiles in (1, 2):
        B.gdn_test_attn_tiles(tiles)
        try:
            res.append(B.gdn_attn_prefill(q, k, v, cu, return_lse=True, out_dtype=F32))
        finally:
            B.gdn_test_attn_tiles(0)
    assert all(torch.equal(a, b) for a, b in zip(*res))


def test_prefill_empty():
    e = torch.empty(0, 4, 64, dtype=BF, device="cuda")
    assert B.gdn_attn_prefill(e, e, e).shape == (0, 4, 64)


@either
@pytest.mark.parametrize("H, Hk, D", [(16, 4, 128), (8, 8, 64)])
def test_prefill_long(H, Hk, D):
    """Many key tiles and many work items at once, against 64-bit products on the GPU."""
    lens = [2500, 1, 1200, 777]
    g = torch.Generator().manual_seed(9)
    T = sum(lens)
    q, k, v = (randn(g, T, h, D).cuda() for h in (H, Hk, Hk))
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    out, lse = B.gdn_attn_prefill(q, k, v, cu.cuda(), return_lse=True, out_dtype=F32)
    for b, e in zip(cu[:-1].tolist(), cu[1:].tolist()):
        kk, vv = (x[b:e].double().repeat_interleave(H // Hk, 1).transpose(0, 1) for x in (k, v))
        s = (q[b:e].double().transpose(0, 1) @ kk.transpose(1, 2)) * D ** -0.5
        s = s.masked_fill(torch.ones(e - b, e - b, device="cuda").triu(1).bool(), float("-inf"))
        w = torch.softmax(s, -1)
        ref, mag, rl = w @ vv, w @ vv.abs(), torch.logsumexp(s, -1)
        d = (out[b:e].double().transpose(0, 1) - ref).abs() - (REL * mag + 1e-6)
        assert d.max().item() <= 0
        assert (lse[b:e].double().t() - rl).abs().max().item() <= 1e-3


# ---------------------------------------------------------------- decode
@pytest.fixture(params=["by rule", "always"])
def prefix_pass(request):
    """The shared prefix with its own pass where the library's rule says so (not at most sizes
    here), and with it at every size."""
    B.gdn_test_attn_prefix(request.param == "always")
    yield
    B.gdn_test_attn_prefix(False)


both = pytest.mark.usefixtures("prefix_pass")


def make_cache(g, lens, Hk, D, page, shared=0, extra=3, fill=float("nan")):
    """A paged cache in scattered page order whose unused rows hold `fill`; returns
    (k_cache, v_cache, table, n_pages) on the CPU."""
    own = [max(0, -(-n // page) - shared // page) for n in lens]
    width = max(1, shared // page + max(own))
    n_pages = shared // page + sum(own) + extra
    perm = torch.randperm(n_pages, generator=g).tolist()
    table = torch.full((len(lens), width), -7, dtype=torch.int32)  # unused entries: no page
    first = [perm.pop() for _ in range(shared // page)]
    kc, vc = (torch.full((n_pages, Hk, page, D), fill, dtype=BF) for _ in range(2))
    for p in first:
        kc[p], vc[p] = randn(g, Hk, page, D), randn(g, Hk, page, D)
    for n, length in enumerate(lens):
        table[n, :len(first)] = torch.tensor(first, dtype=torch.int32)
        for j in range(len(first) * page, length, page):
            p = perm.pop()
            table[n, j // page] = p
            c = min(page, length - j)
            kc[p, :, :c], vc[p, :, :c] = randn(g, Hk, c, D), randn(g, Hk, c, D)
    return kc, vc, table


def check_decode(lens, H, Hk, D, page, nq=1, shared=0, seed=0, scale=None, out_dtype=F32, mul=1.0):
    g = torch.Generator().manual_seed(seed)
    kc, vc, table = make_cache(g, lens, Hk, D, page, shared)
    N = len(lens)
    q = randn(g, N, nq, H, D, mul=mul)
    kv = torch.tensor(lens, dtype=torch.int32)
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    out, lse = B.gdn_attn_decode(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), kv.cuda(), shared,
                                 scale=scale, out_dtype=out_dtype, return_lse=True, status=status)
    assert status.item() == 0
    ref, mag, rl = A.decode(np64(q), np64(kc), np64(vc), table.numpy(), lens, shared, scale)
    close_attention(out, lse, ref, mag, rl)
    return q, kc, vc, table, kv, out


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_pages(page, D):
    check_decode([1, page - 1, page, page + 1, 3 * page + 5, 300], 8, 2, D, page, seed=page)


@pytest.mark.parametrize("H, Hk", [(1, 1), (3, 1), (4, 4), (7, 1), (16, 1), (17, 1), (40, 2), (64, 1)])
def test_decode_groups(H, Hk):
    check_decode([77, 130, 5], H, Hk, 128, 32, seed=H)


@pytest.mark.parametrize("nq, G", [(2, 1), (3, 5), (4, 4), (8, 8), (64, 1), (9, 7), (5, 3)])
def test_decode_several_tokens(nq, G):
    check_decode([nq, nq + 1, 70, 200], 2 * G, 2, 64, 16, nq=nq, seed=nq)


def test_decode_empty_sequences():
    q, kc, vc, table, kv, out = check_decode([0, 40, 0, 1, 0], 4, 2, 128, 16)
    assert (out[[0, 2, 4]] == 0).all()
    check_decode([0], 2, 1, 64, 16)
    check_decode([1, 3, 0], 2, 1, 64, 16, nq=4)  # rows before the sequence's start see nothing


def test_decode_no_rows():
    kc = torch.zeros(3, 2, 16, 64, dtype=BF, device="cuda")
    table, kv = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in ((4, 3), (4,)))
    status = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    q = torch.empty(4, 0, 6, 64, dtype=BF, device="cuda")
    assert B.gdn_attn_decode(q, kc, kc, table, kv, status=status).shape == (4, 0, 6, 64)
    assert status.item() == 0


def test_decode_long_and_uneven():
    """One long axis to split beside many short ones; and a single long sequence."""
    check_decode([9000, 1, 2, 300, 17, 1025], 8, 2, 128, 64, seed=1)
    check_decode([20011], 4, 1, 128, 16, seed=2)
    check_decode([1 + 13 * i % 200 for i in range(97)], 4, 2, 64, 16, seed=3)


@pytest.mark.parametrize("mul", [0.01, 6.0])
def test_decode_score_ranges(mul):
    check_decode([700, 50], 4, 2, 128, 16, mul=mul)


def test_decode_scale_and_bf16_output():
    check_decode([100, 33], 4, 2, 128, 16, scale=0.2)
    check_decode([100, 33], 4, 2, 128, 16, out_dtype=BF)


def test_decode_many_rows():
    """Enough merged rows for one warp each."""
    check_decode([5 + 7 * i % 60 for i in range(130)] + [700] * 5, 8, 2, 64, 16, nq=5, seed=8)


def test_decode_more_units_than_22_bits():
    """Every sequence reads the same few pages, so that the lengths add up without the memory."""
    g = torch.Generator().manual_seed(9)
    N, H, D, page, cols = 4100, 8, 64, 256, 32
    kc, vc = randn(g, 5, H, page, D), randn(g, 5, H, page, D)
    table = torch.randint(0, 5, (N, cols), generator=g, dtype=torch.int32)
    lens = torch.full((N,), cols * page, dtype=torch.int32)
    lens[::7] -= 3
    assert N * H * (cols * page // 64 + 2) > 1 << 22
    q = randn(g, N, H, D)
    out = B.gdn_attn_decode(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), lens.cuda(), out_dtype=F32)
    for n in (0, 1, 2049, N - 1):
        ref, mag, _ = A.decode(np64(q[n:n + 1, None]), np64(kc), np64(vc), table[n:n + 1].numpy(),
                               lens[n:n + 1].tolist())
        close_attention(out[n:n + 1], None, ref, mag, None)


@both
@pytest.mark.parametrize("shared, page", [(16, 16), (128, 16), (112, 16), (384, 128), (256, 256),
                                          (1280, 64)])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_shared_prefix(shared, page, D):
    check_decode([shared + x for x in (1, 0, 40, 17, 300)], 8, 2, D, page, shared=shared, seed=shared)


@both
@pytest.mark.parametrize("N, H, Hk, nq", [(70, 8, 2, 1), (33, 5, 1, 3), (3, 64, 1, 1), (9, 21, 3, 8),
                                          (1, 4, 1, 1), (130, 1, 1, 1)])
def test_decode_shared_prefix_rows(N, H, Hk, nq):
    """Row counts below, at and above a tile of rows, group sizes that do not divide it."""
    check_decode([320 + 5 + 7 * i % 90 for i in range(N)], H, Hk, 64, 32, nq=nq, shared=320, seed=N)


@both
def test_decode_sequences_shorter_than_the_prefix():
    check_decode([200, 64, 0, 1, 320, 319, 257], 4, 2, 128, 64, shared=320, seed=4)
    check_decode([2, 64, 0, 1, 320, 65], 4, 2, 128, 64, nq=3, shared=320, seed=4)


@both
@pytest.mark.parametrize("D", [64, 128])
def test_decode_infinities_where_they_are_seen(D):
    """Infinities and NaN in a prefix that some sequences end inside, and in own tokens."""
    g = torch.Generator().manual_seed(22)
    lens, H, Hk, page, nq, shared = [500, 290, 262, 400, 140, 384], 4, 2, 32, 3, 384
    kc, vc, table = make_cache(g, [max(n, shared) for n in lens], Hk, D, page, shared)
    q = randn(g, len(lens), nq, H, D)
    spots = [(0, 5, 0, 1, float("inf")), (0, 139, 1, 2, -float("inf")), (0, 200, 0, 4, float("inf")),
             (0, 261, 0, 4, -float("inf")), (0, 289, 1, D - 1, float("nan")), (0, 300, 0, 7, float("inf")),
             (0, 498, 1, 8, -float("inf")), (3, 390, 0, 9, float("inf")), (3, 399, 1, 0, float("nan"))]
    for n, t, h, d, x in spots:
        vc[int(table[n, t // page]), h, t % page, d] = x
    kv = torch.tensor(lens, dtype=torch.int32)
    out, lse = B.gdn_attn_decode(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), kv.cuda(), shared,
                                 out_dtype=F32, return_lse=True)
    with np.errstate(invalid="ignore"):
        ref, mag, rl = A.decode(np64(q), np64(kc), np64(vc), table.numpy(), lens, shared)
    same_where_not_finite(out, ref)
    fin = np.isfinite(ref)
    assert (np.abs(np64(out)[fin] - ref[fin]) <= REL * mag[fin] + 1e-6).all() and fin.mean() > 0.5
    assert np.abs(np64(lse) - rl).max() <= 1e-3


@both
def test_decode_long_shared_prefix():
    check_decode([8192 + 1 + i for i in range(20)], 16, 2, 128, 64, shared=8192, seed=5)


@both
def test_decode_shared_equals_unshared():
    """The same batch with and without the hint, each within its tolerance of the oracle."""
    for shared in (0, 512):
        check_decode([512 + 3 * i for i in range(12)], 8, 2, 128, 32, shared=shared, seed=6)


@both
@pytest.mark.parametrize("what", ["nan", "inf", "lowest"])
@pytest.mark.parametrize("shared", [0, 128, 160])
def test_decode_unseen_values_have_no_influence(what, shared):
    """Values that a later token of the batch or a longer sequence sees, and an earlier token
    or a shorter sequence does not: NaN, infinities, the type's lowest value."""
    bad = dict(nan=float("nan"), inf=float("inf"), lowest=torch.finfo(BF).min)[what]
    g = torch.Generator().manual_seed(11)
    lens, H, Hk, D, page, nq = [190, 100, 133, 60], 4, 2, 128, 16, 4
    if shared == 0:
        lens = [190, 100, 50, 3]
    kc, vc, table = make_cache(g, lens, Hk, D, page, shared)
    q = randn(g, 4, nq, H, D)
    kz, vz = kc.clone(), vc.clone()
    spots = [(0, lens[0] - 1), (0, lens[0] - 2), (1, 98), (2, lens[2] - 3)]
    for n, t in spots:  # last tokens; with a prefix, token 98 belongs to all
        p = int(table[n, t // page])
        for c, z in ((kc, kz), (vc, vz)):
            c[p, :, t % page] = bad
            z[p, :, t % page] = 0
    out = B.gdn_attn_decode(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(),
                            torch.tensor(lens, dtype=torch.int32).cuda(), shared, out_dtype=F32)
    ref, mag, rl = A.decode(np64(q), np64(kz), np64(vz), table.numpy(), lens, shared)
    hit = np.zeros((4, nq), bool)  # rows that see a spoilt key
    for n in range(4):
        for i in range(nq):
            mine = [t for m, t in spots if m == n or t < shared]
            hit[n, i] = any(t <= lens[n] - nq + i for t in mine)
    assert hit.any() and not hit.all()
    close_attention(out.view(4 * nq, H, D), None, ref.reshape(4 * nq, H, D),
                    mag.reshape(4 * nq, H, D), None, ~hit.reshape(-1))


@both
def test_decode_bad_pages_and_lengths():
    g = torch.Generator().manual_seed(3)
    kc, vc, table = make_cache(g, [100, 90], 2, 64, 16, fill=0.0)
    table[0, 2], table[1, 0] = 10 ** 6, -3
    q = randn(g, 2, 4, 64)
    for lens, shared, want in (([100, 90], 0, 64), ([100, 90], 48, 64), ([100, 10 ** 9], 0, 64 | 128),
                               ([-5, 90], 0, 64 | 128)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = B.gdn_attn_decode(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(),
                                     torch.tensor(lens, dtype=torch.int32).cuda(), shared,
                                     out_dtype=F32, return_lse=True, status=status)
        assert status.item() == want
        t = np.where(table.numpy() == -7, -1, table.numpy())
        ref, mag, rl = A.decode(np64(q)[:, None], np64(kc), np64(vc), t, lens, shared)
        close_attention(out, lse, ref, mag, rl)


@both
def test_decode_cache_past_32_bit_offsets():
    """Pages whose element offsets pass 2^32."""
    Hk, D, page, n_pages = 8, 128, 256, 18000
    assert n_pages * Hk * page * D > 2 ** 32
    g = torch.Generator().manual_seed(4)
    kc, vc = (torch.empty(n_pages, Hk, page, D, dtype=BF, device="cuda") for _ in range(2))
    table = torch.tensor([[17999, 3, 17500], [9000, 17998, 0]], dtype=torch.int32)
    small = [randn(g, 6, Hk, page, D) for _ in range(2)]
    flat = table.flatten().long().cuda()
    for c, s in zip((kc, vc), small):
        c[flat] = s.cuda()
    q, lens = randn(g, 2, 1, 16, D), [600, 700]
    local = np.arange(6).reshape(2, 3)
    for shared in (0, 512):
        t, loc = table.clone(), local.copy()
        if shared:
            t[1, :2], loc[1, :2] = t[0, :2], loc[0, :2]
        out = B.gdn_attn_decode(q.cuda(), kc, vc, t.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                                shared, out_dtype=F32)
        ref, mag, rl = A.decode(np64(q), np64(small[0]), np64(small[1]), loc, lens, shared)
        close_attention(out, None, ref, mag, rl)


@both
def test_decode_repeatable_other_stream_and_graph():
    g = torch.Generator().manual_seed(7)
    lens = [900, 3, 400, 1500]
    kc, vc, table = (x.cuda() for x in make_cache(g, [1600] * 4, 2, 128, 16, 256, fill=0.5))
    q, kv = randn(g, 4, 8, 128).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    for shared in (0, 256):
        a = B.gdn_attn_decode(q, kc, vc, table, kv, shared)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            b = B.gdn_attn_decode(q, kc, vc, table, kv, shared)
        s.synchronize()
        assert torch.equal(a, b)
        c = torch.zeros_like(a)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            B.gdn_attn_decode(q, kc, vc, table, kv, shared, out=c)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, c)
        kv.copy_(torch.tensor([1600, 299, 0, 1], dtype=torch.int32))
        graph.replay()
        d = B.gdn_attn_decode(q, kc, vc, table, kv, shared)
        torch.cuda.synchronize()
        assert torch.equal(c, d)
        kv.copy_(torch.tensor(lens, dtype=torch.int32))


# ---------------------------------------------------------------- front
def check_front(lens, H, Hk, D, rot, inter=False, x_dtype=BF, out_dtype=BF, page=16, past=None,
                norm=True, cache=True, dense=True, seed=0, lead=0, tail=0, mul=2.0):
    g = torch.Generator().manual_seed(seed)
    N, T = len(lens), lead + sum(lens) + tail
    x = randn(g, T, (H + 2 * Hk) * D, dtype=x_dtype, mul=mul)
    qw, kw = (1 + randn(g, D, dtype=F32, mul=0.2) for _ in range(2)) if norm else (None, None)
    cu = torch.tensor([lead] + lens).cumsum(0).to(torch.int32)
    past = [0] * N if past is None else past
    kv = torch.tensor([p + n for p, n in zip(past, lens)], dtype=torch.int32)
    need = [-(-int(n) // page) for n in kv]
    n_pages, width = sum(need) + 2, max(max(need), 1)
    perm = torch.randperm(n_pages, generator=g).tolist()
    table = torch.full((N, width), -1, dtype=torch.int32)
    for n in range(N):
        for j in range(need[n]):
            table[n, j] = perm.pop()
    kc, vc = (randn(g, n_pages, Hk, page, D, dtype=out_dtype) for _ in range(2))
    rope = rope_table(int(kv.max()) + 1, rot, device="cpu") if rot else None
    dev = lambda t: None if t is None else t.cuda()
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    kd, vd = (dev(kc), dev(vc)) if cache else (None, None)
    bufs = [torch.full((T, h, D), 9.0, dtype=out_dtype, device="cuda") for h in (H, Hk, Hk)]
    q, k, v = B.gdn_attn_front(dev(x), H, Hk, D, dev(qw), dev(kw), rope=dev(rope), interleaved=inter,
                               cu_seqlens=dev(cu), kv_lens=dev(kv),
                               page_table=dev(table) if cache else None, k_cache=kd, v_cache=vd,
                               output_kv=dense, q=bufs[0], k=bufs[1], v=bufs[2],
                               out_dtype=out_dtype, status=status)
    assert status.item() == 0
    ref = A.front(np64(x), H, Hk, D, None if qw is None else np64(qw), None if kw is None else np64(kw),
                  1e-6, None if rope is None else np64(rope), inter, cu.numpy(), kv.numpy(),
                  table.numpy(), np64(kc), np64(vc))
    inside = ref[5]
    assert (k is None) == (not dense)
    pairs = [(q, ref[0]), (k, ref[1]), (v, ref[2])] if dense else [(q, ref[0])]
    for got, want in pairs:
        close_front(got[torch.tensor(inside)], want[inside], out_dtype)
        assert (got[torch.tensor(~inside)] == 9.0).all()
    if cache:
        close_front(kd, ref[3], out_dtype)
        close_front(vd, ref[4], out_dtype)


def close_front(got, want, dtype):
    g = np64(got)
    size = np.abs(want).max(-1, keepdims=True) if want.size else np.abs(want)
    tol = 2e-6 * size + (2.0 ** -8 * np.abs(want) if dtype == BF else 0.0)
    assert (np.abs(g - want) <= tol).all(), np.abs(g - want).max()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D, rot", [(64, 16), (64, 48), (64, 64), (128, 32), (128, 96), (128, 128),
                                    (128, 0)])
def test_front_rotary(D, rot, inter):
    check_front([5, 1, 40], 6, 2, D, rot, inter, past=[7, 300, 0], seed=rot)


@pytest.mark.parametrize("x_dtype, out_dtype", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("D", [64, 128])
def test_front_types(D, x_dtype, out_dtype):
    check_front([33, 2], 5, 1, D, 32, x_dtype=x_dtype, out_dtype=out_dtype, past=[3, 15])


@pytest.mark.parametrize("norm, cache, dense", [(False, True, True), (True, False, True),
                                                (True, True, False), (False, False, True)])
def test_front_parts(norm, cache, dense):
    check_front([20, 11], 4, 2, 128, 64, norm=norm, cache=cache, dense=dense)


@pytest.mark.parametrize("lens, lead, tail", [([1], 0, 0), ([1] * 130, 0, 0), ([1, 0, 1, 0, 3], 0, 0),
                                              ([0, 0, 7], 2, 5), ([0], 0, 4), ([2, 1, 1, 1], 1, 0)])
def test_front_sequences(lens, lead, tail):
    check_front(lens, 4, 2, 128, 64, past=[11 * i % 70 for i in range(len(lens))], lead=lead, tail=tail)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_front_pages(page):
    check_front([page + 3, 2 * page, 5], 3, 1, 64, 64, page=page, past=[page - 1, 0, 2 * page + 7])


def test_front_many_rows():
    """Enough rows for the several-heads-a-group form, a head count it does not divide."""
    check_front([700, 501], 15, 3, 128, 64, seed=2)
    check_front([700, 501], 15, 3, 64, 32, inter=True, x_dtype=F32, out_dtype=F32, seed=2)


def test_front_small_and_zero_rows():
    check_front([3], 2, 1, 128, 64, mul=1e-4)
    check_front([3], 2, 1, 128, 64, mul=0.0)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D, rot", [(64, 16), (128, 0), (128, 32)])
@pytest.mark.parametrize("x_dtype, out_dtype", [(BF, BF), (F32, F32)])
def test_front_elements_that_do_not_turn_are_copied(D, rot, inter, x_dtype, out_dtype):
    """Without a norm, what lies past the rotated part comes out as it went in: an infinity or a
    NaN there changes no other element."""
    g = torch.Generator().manual_seed(31)
    H, Hk, T = 4, 2, 21
    x = randn(g, T, H + 2 * Hk, D, dtype=x_dtype)
    for i, bad in enumerate((float("inf"), -float("inf"), float("nan"))):
        for d in (rot, rot + 5, D - 1):
            x[(5 * i + d) % T, :, d] = bad
    rope = rope_table(T, rot).cuda() if rot else None
    got = B.gdn_attn_front(x.view(T, -1).cuda(), H, Hk, D, rope=rope, interleaved=inter,
                           out_dtype=out_dtype)
    finite = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    ref = A.front(np64(finite).reshape(T, -1), H, Hk, D, rope=None if rope is None else np64(rope),
                  interleaved=inter)
    for y, want, at in zip(got, ref, (0, H, H + Hk)):
        heads = slice(at, at + y.shape[1])
        first = 0 if at == H + Hk else rot
        same = x[:, heads, first:].to(out_dtype).float()
        torch.testing.assert_close(y[..., first:].float().cpu(), same, rtol=0, atol=0, equal_nan=True)
        close_front(y[..., :first], want[..., :first], out_dtype)


@pytest.mark.parametrize("x_dtype", [BF, F32])
@pytest.mark.parametrize("D, rot, inter", [(64, 32, True), (128, 64, False)])
@pytest.mark.parametrize("mul", [1e18, 1e20, 3e29, 5e37])
def test_front_norm_of_large_rows(mul, D, rot, inter, x_dtype):
    """Rows whose squares, or whose sum of squares, pass the largest 32-bit number."""
    check_front([3, 40], 4, 2, D, rot, inter, x_dtype=x_dtype, out_dtype=F32, mul=mul)


@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_front_norm_of_one_large_element(out_dtype):
    """Beside one large element the others go to nothing, in that head alone."""
    g = torch.Generator().manual_seed(32)
    H, Hk, D, T = 4, 2, 128, 9
    x = randn(g, T, H + 2 * Hk, D, dtype=F32)
    for t, big in enumerate((1e15, 1e19, 1e25, 3e38, -3e38)):
        x[t, t % (H + Hk), 7 * t] = big
    qw, kw = (1 + randn(g, D, dtype=F32, mul=0.2) for _ in range(2))
    got = B.gdn_attn_front(x.view(T, -1).cuda(), H, Hk, D, qw.cuda(), kw.cuda(), out_dtype=out_dtype)
    for y, want in zip(got, A.front(np64(x).reshape(T, -1), H, Hk, D, np64(qw), np64(kw))):
        close_front(y, want, out_dtype)


@pytest.mark.parametrize("bad", [float("inf"), -float("inf")])
def test_front_norm_of_an_infinite_element(bad):
    """x / sqrt(mean x^2 + eps) with one x infinite: NaN there, 0 elsewhere in that head; a
    rotation carries the NaN to the element's partner."""
    g = torch.Generator().manual_seed(33)
    H, Hk, D, T, rot = 4, 2, 64, 5, 16
    x = randn(g, T, H + 2 * Hk, D, dtype=F32)
    x[1, 1, 40] = bad  # not rotated
    x[2, H, 3] = bad   # rotated, with element 11
    w = torch.ones(D)
    q, k, v = B.gdn_attn_front(x.view(T, -1).cuda(), H, Hk, D, w.cuda(), w.cuda(),
                               rope=rope_table(T, rot), out_dtype=F32)
    gone = torch.zeros(D, dtype=torch.bool)
    gone[40] = True
    assert torch.equal(torch.isnan(q[1, 1]).cpu(), gone) and (q[1, 1].cpu()[~gone] == 0).all()
    gone[:] = False
    gone[[3, 11]] = True
    assert torch.equal(torch.isnan(k[2, 0]).cpu(), gone) and (k[2, 0].cpu()[~gone] == 0).all()
    assert torch.isnan(q).sum() == 1 and torch.isnan(k).sum() == 2 and torch.isfinite(v).all()


def test_front_without_lengths_and_bad_places():
    g = torch.Generator().manual_seed(5)
    x = randn(g, 40, 4 * 64).cuda()
    rope = rope_table(16, 32)
    kc, vc = (torch.zeros(3, 1, 16, 64, dtype=BF, device="cuda") for _ in range(2))
    table = torch.tensor([[1, 99]], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k, v = B.gdn_attn_front(x, 2, 1, 64, rope=rope, page_table=table, k_cache=kc, v_cache=vc,
                               status=status)
    assert status.item() == 64 | 128  # page 99; positions past both tables
    assert torch.equal(kc[1, 0], k[:16, 0]) and torch.equal(vc[1, 0], v[:16, 0])
    assert (kc[[0, 2]] == 0).all() and (vc[[0, 2]] == 0).all()
    ref = A.front(np64(x), 2, 1, 64, rope=np64(rope))
    close_front(q, ref[0], BF)  # positions past the table use its last row
    kv = torch.tensor([20], dtype=torch.int32, device="cuda")  # 40 tokens, 20 of them before the start
    B.gdn_attn_front(x, 2, 1, 64, rope=rope_table(64, 32), kv_lens=kv, page_table=table, k_cache=kc,
                     v_cache=vc, status=status)
    assert status.item() & 128
    B.gdn_attn_front(x, 2, 1, 64, cu_seqlens=torch.tensor([0, 30, 20, 45], dtype=torch.int32).cuda(),
                     status=status)
    assert status.item() == 1


def test_front_graph_and_stream():
    g = torch.Generator().manual_seed(6)
    x = randn(g, 64, 6 * 128).cuda()
    rope = rope_table(64, 64)
    a = B.gdn_attn_front(x, 4, 1, 128, rope=rope)
    out = [torch.zeros_like(t) for t in a]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.gdn_attn_front(x, 4, 1, 128, rope=rope, q=out[0], k=out[1], v=out[2])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(s, t) for s, t in zip(a, out))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = B.gdn_attn_front(x, 4, 1, 128, rope=rope, stream=s)
    s.synchronize()
    assert all(torch.equal(u, t) for u, t in zip(a, b))


@pytest.mark.parametrize("call", ["front", "prefill", "decode"])
def test_memory_waits_for_the_calls_stream(call):
    """What a call allocates, its workspace included, is not free for other work while the
    stream that it was given still has the call before it."""
    x = torch.zeros(8, 6 * 128, dtype=BF, device="cuda")
    q, k = (torch.zeros(8, h, 128, dtype=BF, device="cuda") for h in (4, 1))
    kc = torch.zeros(3, 1, 16, 128, dtype=BF, device="cuda")
    table = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    kv = torch.full((8,), 20, dtype=torch.int32, device="cuda")
    run = {"front": lambda s: B.gdn_attn_front(x, 4, 1, 128, stream=s),
           "prefill": lambda s: B.gdn_attn_prefill(q, k, k, stream=s),
           "decode": lambda s: B.gdn_attn_decode(q, kc, kc, table, kv, stream=s)}[call]

    def waiting():
        return [b["size"] for seg in torch.cuda.memory_snapshot() for b in seg["blocks"]
                if b["state"] == "active_awaiting_free" or b["state"] == "active_pending_free"]

    s = torch.cuda.Stream()
    run(None)
    torch.cuda.synchronize()
    assert not waiting()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)  # about 0.1 s
    out = run(s)
    held = len(waiting())
    assert held == (1 if call == "decode" else 0)
    del out
    assert len(waiting()) == held + (3 if call == "front" else 1)
    s.synchronize()
    torch.cuda.empty_cache()
    assert not waiting()


def stream_call(call):
    """A call with its outputs to be allocated, or with them given: run(stream, **outputs), the
    outputs' names and shapes, and the bytes of a workspace."""
    g = torch.Generator().manual_seed(41)
    x = randn(g, 8, 6 * 128).cuda()
    q, k = (randn(g, 8, h, 128).cuda() for h in (4, 1))
    kc = randn(g, 3, 1, 16, 128).cuda()
    table = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    kv = torch.full((8,), 20, dtype=torch.int32, device="cuda")
    if call == "front":
        return (lambda s, **kw: B.gdn_attn_front(x, 4, 1, 128, stream=s, **kw),
                dict(q=(8, 4, 128), k=(8, 1, 128), v=(8, 1, 128)), 0)
    if call == "prefill":
        return lambda s, **kw: (B.gdn_attn_prefill(q, k, k, stream=s, **kw),), dict(out=(8, 4, 128)), 0
    size = B.gdn_attn_workspace_size(B.make_attn_desc(8, 8, 4, 1, 128, page_size=16, n_pages=3, max_pages=2))
    return (lambda s, **kw: (B.gdn_attn_decode(q, kc, kc, table, kv, stream=s, **kw),),
            dict(out=(8, 4, 128)), size)


@pytest.mark.parametrize("call", ["front", "prefill", "decode"])
def test_memory_is_free_before_the_calls_stream_uses_it(call):
    """Memory that the current stream's queued work still writes is given back and allocated
    again by a call on another stream: the call comes after that work."""
    run, shapes, size = stream_call(call)
    want = run(None)
    s, here = torch.cuda.Stream(), torch.cuda.current_stream()
    run(s)  # (first use of the stream)
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)  # about 0.2 s
    tmp = [torch.empty(shape, dtype=BF, device="cuda") for shape in shapes.values()]
    tmp += [torch.empty(size, dtype=torch.uint8, device="cuda")] if size else []
    for t in tmp:
        t.view(torch.uint8).fill_(255)
    places = [t.data_ptr() for t in tmp]
    del tmp, t
    got = run(s)
    assert not here.query() and not s.query()  # the sleep runs, and the call waits for it
    torch.cuda.synchronize()
    assert {t.data_ptr() for t in got} & set(places)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("call", ["front", "prefill", "decode"])
def test_a_call_that_allocates_nothing_waits_for_its_own_stream_only(call):
    run, shapes, size = stream_call(call)
    want = run(None)
    given = {n: torch.zeros(shape, dtype=BF, device="cuda") for n, shape in shapes.items()}
    if size:
        given["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    s, here = torch.cuda.Stream(), torch.cuda.current_stream()
    run(s, **given)
    torch.cuda.synchronize()
    for t in given.values():
        t.zero_()
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)
    got = run(s, **given)
    s.synchronize()
    assert not here.query()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("call", ["front", "prefill", "decode"])
def test_memory_between_captured_and_other_streams(call):
    """A call on a stream that joined the capture is captured with what it allocates; where only
    one of the two streams is captured, it is refused, unless all is given."""
    run, shapes, size = stream_call(call)
    want = run(None)
    s, lone = torch.cuda.Stream(), torch.cuda.Stream()
    x = torch.zeros(4, device="cuda")
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        x += 1
        s.wait_stream(torch.cuda.current_stream())
        got = run(s)
        torch.cuda.current_stream().wait_stream(s)
        with pytest.raises(ValueError, match="captured"):
            run(lone)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    given = {n: torch.zeros(shape, dtype=BF, device="cuda") for n, shape in shapes.items()}
    if size:
        given["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(other, stream=s):
        with torch.cuda.stream(lone):
            with pytest.raises(ValueError, match="captured"):
                run(s)
            run(s, **given)
    other.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, given[n]) for a, n in zip(want, shapes))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("call", ["prefill", "decode"])
@pytest.mark.parametrize("item", [0, 1, 2])
def test_a_wait_that_runs_out_is_reported_and_leaves_the_next_call_right(call, D, item):
    """The testing hook has the warp that issues the products wait, before a CTA's first, second
    or third work item, for an event that never happens: the call returns with GDN_DEV_TIMEOUT,
    and with the hook off the same call on the same buffers gives its results again."""
    g = torch.Generator().manual_seed(51)
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    if call == "prefill":
        q, k, v = (randn(g, 20000, h, D).cuda() for h in (16, 4, 4))
        cu = torch.tensor([0, 7000, 7001, 20000], dtype=torch.int32, device="cuda")
        run = lambda out: B.gdn_attn_prefill(q, k, v, cu, out=out, status=status)
    else:
        shared, N, Hk = 1024, 700, 4  # 700 items of the prefix: 175 pairs of row tiles x 4
        kc, vc = (randn(g, 64, Hk, 64, D).cuda() for _ in range(2))
        table = torch.randint(0, 64, (N, 20), generator=g, dtype=torch.int32)
        table[:, :16] = table[0, :16]
        q, table = randn(g, N, 4, 64, D).cuda(), table.cuda()
        kv = (1024 + torch.randint(5, 250, (N,), generator=g)).to(torch.int32).cuda()
        run = lambda out: B.gdn_attn_decode(q, kc, vc, table, kv, shared, out=out, status=status)
    want = torch.zeros_like(q)
    out = torch.zeros_like(q)
    B.gdn_test_attn_prefix(True)
    try:
        run(want)
        assert status.item() == 0
        B.gdn_test_attn_timeout(256, item)
        run(out)
        assert status.item() & 8
        B.gdn_test_attn_timeout(0)
        run(out)
        assert status.item() == 0 and torch.equal(out, want)
    finally:
        B.gdn_test_attn_timeout(0)
        B.gdn_test_attn_prefix(False)


# ---------------------------------------------------------------- together
def test_prompt_then_decode_equals_a_longer_prompt():
    """front + prefill of a prompt, then front + decode of the next tokens, give the rows that
    one longer prompt gives."""
    g = torch.Generator().manual_seed(8)
    H, Hk, D, L, more = 8, 2, 128, 150, 5
    x = randn(g, L + more, (H + 2 * Hk) * D).cuda()
    w = torch.ones(D, device="cuda")
    rope = rope_table(256, 64)
    q, k, v = B.gdn_attn_front(x, H, Hk, D, w, w, rope=rope)
    want = np64(B.gdn_attn_prefill(q, k, v, out_dtype=F32))
    table = torch.arange(16, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    kc, vc = (torch.zeros(16, Hk, 16, D, dtype=BF, device="cuda") for _ in range(2))
    for b, e in ((0, L), (L, L + 1), (L + 1, L + more)):
        kv = torch.tensor([e], dtype=torch.int32, device="cuda")
        q1, k1, v1 = B.gdn_attn_front(x[b:e], H, Hk, D, w, w, rope=rope, kv_lens=kv, page_table=table,
                                      k_cache=kc, v_cache=vc)
        if b == 0:
            got = B.gdn_attn_prefill(q1, k1, v1, out_dtype=F32)
        else:
            got = B.gdn_attn_decode(q1[None], kc, vc, table, kv, out_dtype=F32)[0]
        # both sides round their weights to bf16: twice the oracle's tolerance, |v| < 6
        assert np.abs(np64(got) - want[b:e]).max() <= 2 * REL * 6


@both
@pytest.mark.parametrize("document, own", [(512, 37), (200, 5), (64, 1)])
def test_example_layer(document, own):
    """The example's serving loop against its one-prompt form; both sides round their weights
    to bf16: twice the oracle's tolerance, |v| < 6."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "attention_layer.py")
    spec = importlib.util.spec_from_file_location("attention_layer", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert m.main(document=document, own=own) <= 2 * REL * 6


@both
def test_outputs_and_workspace_stay_in_their_bounds():
    """Outputs lie between guard rows that no call touches."""
    g = torch.Generator().manual_seed(12)
    H, Hk, D, T = 6, 2, 64, 77
    buf = torch.full((T + 8, H, D), 3.0, dtype=BF, device="cuda")
    q, k, v = (randn(g, T, h, D).cuda() for h in (H, Hk, Hk))
    B.gdn_attn_prefill(q, k, v, out=buf[4:-4])
    assert (buf[:4] == 3.0).all() and (buf[-4:] == 3.0).all()
    kc, vc, table = (x.cuda() for x in make_cache(g, [90, 33], Hk, D, 16, fill=0.0))
    kv = torch.tensor([90, 33], dtype=torch.int32, device="cuda")
    out = torch.full((10, H, D), 3.0, dtype=BF, device="cuda")
    n = B.gdn_attn_workspace_size(B.make_attn_desc(2, 2, H, Hk, D, page_size=16, n_pages=kc.shape[0],
                                                   max_pages=table.shape[1]))
    work = torch.full((n + 8192,), 7, dtype=torch.uint8, device="cuda")
    for shared in (0, 16):
        t = table.clone()
        t[:, :shared // 16] = t[0, :shared // 16]
        B.gdn_attn_decode(q[:2].contiguous(), kc, vc, t, kv, shared, out=out[4:6],
                          workspace=work[4096:4096 + n])
        assert (out[:4] == 3.0).all() and (out[6:] == 3.0).all()
        assert (work[:4096] == 7).all() and (work[4096 + n:] == 7).all()
