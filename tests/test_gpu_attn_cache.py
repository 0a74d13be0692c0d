"""The long-conversation operators through the C ABI against the fp64 oracle.

Tolerances, derived before the first run:
  - append and evict: every step is exact or one rounding of an exact value, so bytes, scales,
    weights, lengths and places are the oracle's (only a rounding to a scale that is no power of
    two, of a value computed in fp32, may fall on the other side of a tie: those tests allow one
    step of e4m3).
  - attention: each weight may be rounded to bf16 (relative 2^-8 at most), which moves an output
    by at most 2^-8 sum_j w_ij |v_j|; scores and exp add less than 2^-11 of the same sum at these
    inputs. A bf16 output adds 2^-8 |o|. lse: 1e-3 as for the bf16 cache.
    Over a cache in 8 bits, weight times scale, w_j s_j, is rounded to fp16 against a reference r of
    its row: relatively by 2^-12 (within the 2^-8 above), or, where it becomes subnormal, by 2^-25 r.
    r is set to 2^-7 of the largest w_j s_j so far and only grows, so that r <= 2^-7 max_j w_j s_j,
    and an output moves by at most 2^-32 max_j(w_j s_j) sum_j |e_j|, e_j being the e4m3 value: it
    counts where the keys of large weight have a value of 0.
  - weights: fp32 throughout. A score is off by at most (D + 8) 2^-24 scale sum |q k|, a row's lse by
    as much, and exp of their difference by that amount relatively, and 2^-19 for exp itself and the
    sums. A sum that is added to rounds by 2^-24 of it.
  - front: fp32 arithmetic of about ten roundings, 2e-6 relative to the pair's size; bf16 2^-8.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_chunk_gb300 import binding as B
from gated_delta_rule_chunk_gb300.rope import rope_table
from oracle import attention as A
from oracle import attention_cache as C

pytestmark = pytest.mark.gpu

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
REL = 2.0 ** -8 + 2.0 ** -11


def randn(g, *shape, dtype=BF, mul=1.0):
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * mul).to(dtype)


def np64(x):
    return x.detach().double().cpu().numpy()


def as_bytes(x):
    return x.detach().view(torch.uint8).cpu().numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def new_status():
    return torch.full((1,), -1, dtype=torch.int32, device="cuda")


def pages_for(g, counts, extra=0):
    """A table [N, max(counts)] of scattered pages (-1 past a sequence's), and the pages in all."""
    perm = torch.randperm(sum(counts) + extra, generator=g).tolist()
    table = torch.full((len(counts), max(max(counts), 1)), -1, dtype=torch.int32)
    for n, c in enumerate(counts):
        for i in range(c):
            table[n, i] = perm.pop()
    return table, sum(counts) + extra, perm


def random_cache8(g, n_pages, Hk, page, D, spread=3, power=True):
    """Bytes of any finite value, scales of different sizes."""
    b = torch.randint(0, 256, (n_pages, Hk, page, D), generator=g, dtype=torch.uint8)
    b[(b & 127) == 127] = 126
    s = torch.exp2(torch.randint(-spread, spread + 1, (n_pages, Hk, page // 16), generator=g).float() - 8)
    if not power:
        s = s * (0.5 + torch.rand(s.shape, generator=g))
    return b, s


def values8(b, s):
    return C.held(b.numpy(), s.numpy())


# ---------------------------------------------------------------- append
def check_append(lens, pasts, Hk, D, page, dtype=BF, seed=0, lead=0, tail=0, spoil=None, kv=True, old_scale=None):
    g = torch.Generator().manual_seed(seed)
    T = lead + sum(lens) + tail
    k = randn(g, T, Hk, D, dtype=dtype) * torch.exp2(torch.randint(-6, 7, (T, Hk, 1), generator=g).to(dtype))
    v = randn(g, T, Hk, D, dtype=dtype, mul=5.0)
    if spoil:
        spoil(k, v)
    ends = [p + n for p, n in zip(pasts, lens)]
    table, n_pages, _ = pages_for(g, [-(-e // page) for e in ends], 1)
    kb, ks = random_cache8(g, n_pages, Hk, page, D, old_scale or 3)
    vb, vs = random_cache8(g, n_pages, Hk, page, D, old_scale or 3)
    cu = np.cumsum([lead] + lens)
    dev = [x.cuda() for x in (kb, vb, ks, vs)]
    status = new_status()
    for _ in range(2):  # a second call changes nothing
        B.gdn_attn_append8(k.cuda(), v.cuda(), dev[0].view(F8), dev[1].view(F8), dev[2], dev[3],
                           table.cuda(), kv_lens=i32(ends) if kv else None, cu_seqlens=i32(cu.tolist()),
                           status=status)
        assert status.item() == 0
        for x, b, s, got_b, got_s in ((k, kb, ks, dev[0], dev[2]), (v, vb, vs, dev[1], dev[3])):
            want_b, want_s = C.append8(np64(x), b.numpy(), s.numpy(), table.numpy(), ends if kv else None, cu)
            assert np.array_equal(got_s.cpu().numpy(), want_s)
            assert C.same_bytes(as_bytes(got_b), want_b).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_append_pages(page, D):
    check_append([page + 5, 1, 40], [0, page - 1, 7], 2, D, page, seed=page)


@pytest.mark.parametrize("lens, pasts", [
    ([1], [0]), ([1], [15]), ([1], [16]), ([1], [31]), ([1] * 40, list(range(40))), ([15], [1]), ([17], [15]),
    ([33], [0]), ([2, 0, 0, 3, 1], [30, 4, 0, 15, 16]), ([0, 0, 70], [3, 0, 9]), ([1, 1, 300], [5, 6, 7]),
    ([2] * 20, [15] * 20),
])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_lengths(lens, pasts, dtype):
    check_append(lens, pasts, 3, 128, 32, dtype=dtype, seed=sum(lens), lead=2, tail=5)


@pytest.mark.parametrize("Hk", [1, 5, 16])
def test_append_heads(Hk):
    check_append([20, 1, 9], [3, 40, 0], Hk, 64, 16, seed=Hk)


def test_append_without_lengths():
    check_append([37, 5], [0, 0], 2, 128, 16, kv=False)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_sizes_at_the_limits(dtype):
    """Zeros, the smallest and the largest numbers, and a maximum on either side of 448 s."""
    def spoil(k, v):
        k[0:16] = 0.0
        k[16:32] = 2.0 ** -126
        k[32:48] = torch.finfo(dtype).max
        k[48:64] = 1.75
        k[64:80] = 1.765625
        v[0:16, :, 0] = 1e-30
        v[16:32] *= 2.0 ** 60
        v[40] = 0.0
    check_append([90], [16], 2, 64, 32, dtype=dtype, spoil=spoil)
    check_append([90], [3], 2, 64, 32, dtype=dtype, spoil=spoil, old_scale=20)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_append_what_is_not_finite_is_nan_alone(bad):
    def spoil(k, v):
        k[3, 0, 5] = bad
        v[17:33] = bad
    check_append([40], [2], 2, 64, 16, spoil=spoil)


def test_append_grown_scales_round_again():
    """Token by token, each larger than the one before: the oracle's same chain of roundings."""
    g = torch.Generator().manual_seed(3)
    D, Hk = 128, 2
    x = randn(g, 20, Hk, D) * torch.exp2(torch.arange(20)).to(BF)[:, None, None]
    table = torch.tensor([[1, 0]], dtype=torch.int32)
    kb, ks = random_cache8(g, 2, Hk, 16, D)
    dev = [kb.cuda(), kb.cuda(), ks.cuda(), ks.cuda()]
    b, s = kb.numpy(), ks.numpy()
    for t in range(20):
        B.gdn_attn_append8(x[t:t + 1].cuda(), x[t:t + 1].cuda(), dev[0].view(F8), dev[1].view(F8), dev[2],
                           dev[3], table.cuda(), kv_lens=i32([t + 1]))
        b, s = C.append8(np64(x[t:t + 1]), b, s, table.numpy(), [t + 1])
    for i in (0, 1):
        assert C.same_bytes(as_bytes(dev[i]), b).all() and np.array_equal(dev[2 + i].cpu().numpy(), s)


def test_append_over_scales_that_are_no_powers_of_two():
    """A block's scale that another program chose stays while it is large enough; one step of e4m3."""
    g = torch.Generator().manual_seed(4)
    kb, ks = random_cache8(g, 1, 1, 16, 64)
    ks[:] = 0.0123
    x = randn(g, 3, 1, 64)
    dev = [kb.cuda(), kb.cuda(), ks.cuda(), ks.cuda()]
    B.gdn_attn_append8(x.cuda(), x.cuda(), dev[0].view(F8), dev[1].view(F8), dev[2], dev[3], i32([[0]]),
                       kv_lens=i32([9]))
    want, s = C.append8(np64(x), kb.numpy(), ks.numpy(), np.array([[0]]), [9])
    assert np.array_equal(dev[2].cpu().numpy(), s) and s.item() == ks.item()
    a, b = C.VALUES[as_bytes(dev[0])], C.VALUES[want]
    assert (np.abs(a - b) <= 2.0 ** -3 * np.abs(b)).all() and (a != b).mean() < 0.01


def test_append_places_that_do_not_exist():
    g = torch.Generator().manual_seed(5)
    kb, ks = random_cache8(g, 3, 2, 16, 64)
    table = i32([[0, 7, 2], [-1, 1, 1]])
    x = randn(g, 60, 2, 64).cuda()
    dev = [kb.cuda(), kb.cuda(), ks.cuda(), ks.cuda()]
    status = new_status()
    cu, lens = i32([0, 50, 60]), i32([52, 8])  # sequence 0 passes the table's end, 1 begins at -2
    B.gdn_attn_append8(x, x, dev[0].view(F8), dev[1].view(F8), dev[2], dev[3], table, kv_lens=lens,
                       cu_seqlens=cu, status=status)
    assert status.item() == 64 | 128
    want, s = C.append8(np64(x[:50]), kb.numpy(), ks.numpy(), table.cpu().numpy()[:1], [52])
    assert C.same_bytes(as_bytes(dev[0]), want).all() and np.array_equal(dev[2].cpu().numpy(), s)
    B.gdn_attn_append8(x, x, dev[0].view(F8), dev[1].view(F8), dev[2], dev[3], table, kv_lens=lens,
                       cu_seqlens=i32([0, 70, 60]), status=status)
    assert status.item() & 1


@pytest.mark.parametrize("cu", [[0, 40, 90], [0, 61], [-3, 20, 90, 60], [0, 2, 2 ** 31 - 1]])
def test_append_sequences_that_pass_the_rows(cu):
    """What lies behind k and v (NaN here) does not reach the cache."""
    g = torch.Generator().manual_seed(6)
    N, T, Hk, D = len(cu) - 1, 60, 2, 64
    kb, ks = random_cache8(g, 8 * N, Hk, 16, D)
    x = torch.full((T + 40, Hk, D), float("nan"), dtype=BF)
    x[:T] = randn(g, T, Hk, D)
    table = torch.arange(8 * N, dtype=torch.int32).reshape(N, 8)
    for dtype in (BF, F32):
        k = x.to(dtype).cuda()[:T]
        dev = [kb.cuda(), kb.cuda(), ks.cuda(), ks.cuda()]
        status = new_status()
        B.gdn_attn_append8(k, k, dev[0].view(F8), dev[1].view(F8), dev[2], dev[3], table.cuda(), cu_seqlens=i32(cu),
                           status=status)
        assert status.item() & 1
        for b, s in ((dev[0], dev[2]), (dev[1], dev[3])):
            assert np.isfinite(C.VALUES[as_bytes(b)]).all() and torch.isfinite(s).all()
        if 0 <= cu[1] <= T and cu[0] == 0:
            want, s = C.append8(np64(x[:cu[1]]), kb.numpy(), ks.numpy(), table.numpy()[:1])
            assert C.same_bytes(as_bytes(dev[0])[:8], want[:8]).all()
            assert np.array_equal(dev[2].cpu().numpy()[:8], s[:8])


# ---------------------------------------------------------------- decode
def close(out, lse, ref, mag, ref_lse, floor=0.0):
    o = np64(out).reshape(ref.shape)
    tol = REL * mag + (2.0 ** -8 * np.abs(ref) if out.dtype == BF else 0.0) + 1e-6 * mag + floor
    bad = ~(np.abs(o - ref) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], o[bad][:5], ref[bad][:5], tol[bad][:5])
    got, want = np64(lse).reshape(ref_lse.shape), ref_lse
    assert np.array_equal(np.isneginf(got), np.isneginf(want))
    fin = np.isfinite(want)
    assert np.abs(got[fin] - want[fin]).max(initial=0.0) <= 1e-3


def fp16_floor(q, keys, vb, vs, table, lens, shared=0, scale=None):
    """2^-32 max_j(w_j s_j) sum_j |e_j| for rows q [N, n_q, H, D] over keys' values, bytes and scales."""
    N, nq, H, D = q.shape
    Hk, page = keys.shape[1:3]
    e = np.abs(C.VALUES[vb.numpy()])
    s = np.repeat(vs.double().numpy(), 16, 2)[..., None]
    floor = np.zeros(q.shape)
    for n in range(N):
        length = min(max(lens[n], 0), table.shape[1] * page)
        last = np.arange(length - nq, length)
        for h in range(H):
            k, ev, sv = (A.gather(x, table.numpy(), n, length, h * Hk // H, page, shared) for x in (keys, e, s))
            w = C.row_weights(q[n, :, h], k, last, D ** -0.5 if scale is None else scale)
            for i in range(nq):
                seen = max(last[i] + 1, 0)
                if seen:
                    floor[n, i, h] = 2.0 ** -32 * (w[i, :seen] * sv[:seen, 0]).max() * ev[:seen].sum(0)
    return floor


def weight_slack(q, keys, D, scale):
    """Relative error of a weight, from the largest sum of |q k| there is."""
    most = scale * np.abs(np64(q)).sum(-1).max() * np.abs(keys).max()
    most = min(most, scale * np.sqrt((np64(q) ** 2).sum(-1).max() * (keys ** 2).sum(-1).max()))
    return 2 * (D + 8) * 2.0 ** -24 * most + 2.0 ** -19


def run_decode(lens, H, Hk, D, page, nq=1, bits=8, weights=False, seed=0, mul=1.0, scale=None,
               out_dtype=F32, shared=0, power=True, spread=1, spoil=None):
    g = torch.Generator().manual_seed(seed)
    N = len(lens)
    q = randn(g, *((N, H, D) if nq == 1 else (N, nq, H, D)), mul=mul)
    counts = [-(-max(n, 0) // page) for n in lens]
    table, n_pages, _ = pages_for(g, counts, 1)
    if shared:
        table[:, :shared // page] = table[max(range(N), key=lambda n: counts[n]), :shared // page]
    if bits == 8:
        kb, ks = random_cache8(g, n_pages, Hk, page, D, spread, power)
        vb, vs = random_cache8(g, n_pages, Hk, page, D, spread, power)
        kv, vv = values8(kb, ks), values8(vb, vs)
    else:
        kb, vb, ks, vs = randn(g, n_pages, Hk, page, D), randn(g, n_pages, Hk, page, D), None, None
        kv, vv = np64(kb), np64(vb)
    w = torch.rand(n_pages, Hk, page, generator=g) * 3 if weights else None
    if spoil:
        kv, vv = spoil(q, kb, vb, ks, vs, table, w, kv, vv)
    dev = lambda x: None if x is None else x.cuda()
    k_dev, v_dev = dev(kb), dev(vb)
    if bits == 8:
        k_dev, v_dev = k_dev.view(F8), v_dev.view(F8)
    w_dev, status = dev(w), new_status()
    out, lse = B.gdn_attn_decode(q.cuda(), k_dev, v_dev, table.cuda(), i32(lens), shared_len=shared,
                                 scale=scale, out_dtype=out_dtype, return_lse=True, status=status,
                                 k_scale=dev(ks), v_scale=dev(vs), weights=w_dev)
    assert status.item() == 0
    q4 = np64(q).reshape(N, nq, H, D)
    ref, mag, rl = A.decode(q4, kv, vv, table.numpy(), lens, shared, scale)
    floor = fp16_floor(q4, kv, vb, vs, table, lens, shared, scale) if bits == 8 else 0.0
    close(out, lse, ref, mag, rl, floor)
    if weights:
        want = C.decode_weights(q4, kv, table.numpy(), lens, w.numpy(), scale)
        seen = [kv[int(table[n, j // page]), :, j % page] for n in range(N) for j in range(lens[n])]
        keys = np.array(seen) if seen else np.zeros((1, 1, D))
        tol = weight_slack(q, keys, D, scale or D ** -0.5) * np.abs(want) + 2.0 ** -22 * np.abs(want) + 1e-9
        got = np64(w_dev)
        bad = ~((np.abs(got - want) <= tol) | (np.isnan(got) & np.isnan(want)))
        assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], tol[bad][:5])


FORMS = pytest.mark.parametrize("bits, weights", [(8, False), (8, True), (16, True)])


@FORMS
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_decode_pages(page, D, bits, weights):
    run_decode([1, page - 1, page, page + 1, 3 * page + 7], 4, 2, D, page, bits=bits, weights=weights, seed=page)


@FORMS
@pytest.mark.parametrize("H, Hk", [(1, 1), (3, 3), (3, 1), (5, 1), (6, 2), (7, 1), (16, 2), (24, 2), (33, 1), (64, 1)])
def test_decode_groups(H, Hk, bits, weights):
    run_decode([70, 1, 150], H, Hk, 128, 16, bits=bits, weights=weights, seed=H)


@FORMS
@pytest.mark.parametrize("nq, G", [(2, 1), (3, 5), (4, 4), (5, 3), (8, 8), (16, 4), (64, 1)])
def test_decode_several_tokens(nq, G, bits, weights):
    run_decode([nq, nq + 1, 100, nq + 15, 257], 2 * G, 2, 64, 32, nq=nq, bits=bits, weights=weights, seed=nq)


@pytest.mark.parametrize("rows", [17, 24, 25, 32, 33, 40, 48, 49])
@pytest.mark.parametrize("D", [64, 128])
def test_decode8_rows_of_a_key_head(rows, D):
    """Either side of each change of the warps' tiles, with one token and with several."""
    run_decode([300, 17, 0, 1000], rows, 1, D, 32, weights=True, seed=rows)
    nq = next(n for n in (8, 7, 5, 3, 1) if rows % n == 0)
    run_decode([300, 2, 129, 700], rows // nq * 2, 2, D, 16, nq=nq, seed=rows)


@FORMS
def test_decode_fewer_keys_than_rows_and_none(bits, weights):
    run_decode([0, 5, 2, 0, 1, 33], 2, 1, 64, 16, nq=4, bits=bits, weights=weights)
    run_decode([0, 0], 4, 2, 128, 16, bits=bits, weights=weights)


@FORMS
def test_decode_long_and_uneven(bits, weights):
    run_decode([3000, 1, 777, 0, 64, 2049], 8, 2, 128, 64, bits=bits, weights=weights)
    run_decode([5000], 6, 2, 64, 16, nq=3, bits=bits, weights=weights)


@FORMS
@pytest.mark.parametrize("mul", [0.01, 4.0, 16.0])
def test_decode_score_ranges(mul, bits, weights):
    run_decode([385, 90], 4, 2, 128, 32, bits=bits, weights=weights, mul=mul)


@FORMS
def test_decode_scale_and_bf16_output(bits, weights):
    run_decode([200, 31], 4, 1, 128, 16, scale=0.02, bits=bits, weights=weights)
    run_decode([200, 31], 4, 1, 64, 16, out_dtype=BF, bits=bits, weights=weights)


@FORMS
def test_decode_many_sequences(bits, weights):
    run_decode([1 + 37 * i % 90 for i in range(200)], 4, 2, 64, 16, bits=bits, weights=weights)


def test_decode8_scales_of_any_size():
    """Blocks whose scales differ by many powers of two: the small ones count where the large have
    no weight, and scales that are no powers of two."""
    run_decode([400, 100], 4, 2, 128, 16, power=False)

    def spoil(q, kb, vb, ks, vs, table, w, kv, vv):
        # values of the first half of a sequence 2^40 times those of the second, and the keys of the
        # first half score far below the others'
        q[:] = 1.0
        kb[:] = 0x38  # 1.0
        ks[:] = 2.0 ** -6
        vs[:] = 2.0 ** -30
        for i in range(table.shape[1] // 2):
            p = int(table[0, i])
            kb[p] = 0xB8  # -1.0
            ks[p] = 2.0
            vs[p] = 2.0 ** 10
        return values8(kb, ks), values8(vb, vs)
    run_decode([320], 4, 2, 128, 16, spoil=spoil)

    def extreme(q, kb, vb, ks, vs, table, w, kv, vv):
        ks[:] = 2.0 ** -100
        vs[:] = 2.0 ** 100
        vs[::2] = 2.0 ** -100
        q[:, 0] *= 2.0 ** 90
        return values8(kb, ks), values8(vb, vs)
    run_decode([100, 33], 2, 1, 64, 16, spoil=extreme)


def test_decode8_zero_scales():
    def spoil(q, kb, vb, ks, vs, table, w, kv, vv):
        ks[:] = 0.0
        vs[0] = 0.0
        return values8(kb, ks), values8(vb, vs)
    run_decode([100, 33], 2, 1, 64, 16, spoil=spoil, weights=True)


def test_decode8_large_queries():
    """Queries past fp16's range, and rows of very different sizes."""
    def spoil(q, kb, vb, ks, vs, table, w, kv, vv):
        q[:] = q * torch.tensor([2.0 ** 20, 1.0, 2.0 ** -20, 2.0 ** 100]).to(BF)[None, :, None]
        ks[:] = 2.0 ** -28
        ks[1] = 2.0 ** -120
        return values8(kb, ks), values8(vb, vs)
    # (with this scale the last head's scores are of ordinary size, the others' nearly 0)
    run_decode([64, 17], 4, 1, 64, 16, spoil=spoil, scale=2.0 ** -80)


@FORMS
@pytest.mark.parametrize("nq", [1, 4])
def test_decode_what_is_not_seen_has_no_influence(nq, bits, weights):
    """Rows past a sequence's length, in its last page: NaN elements, scales and weights; and stale
    weights of the call's own tokens."""
    lens = [5, 40, 16]

    def spoil(q, kb, vb, ks, vs, table, w, kv, vv):
        for n, length in enumerate(lens):
            p, r = int(table[n, (length - 1) // 32]), (length - 1) % 32 + 1
            for x in (kb, vb):
                x[p, :, r:] = 0x7F if bits == 8 else float("nan")
            if bits == 8:
                ks[p, :, (r + 15) // 16:] = float("nan")
                vs[p, :, (r + 15) // 16:] = float("inf")
            if w is not None:
                w[p, :, r:] = float("nan")
                for j in range(length - min(nq, length), length):
                    w[int(table[n, j // 32]), :, j % 32] = float("inf")
        return kv, vv
    run_decode(lens, 4, 2, 64, 32, nq=nq, bits=bits, weights=weights, spoil=spoil)


def test_decode8_later_rows_values_that_are_nan():
    """Row i does not see the tokens behind it: a NaN key or value there reaches the rows after only."""
    g = torch.Generator().manual_seed(9)
    kb, ks = random_cache8(g, 3, 1, 16, 64)
    vb, vs = random_cache8(g, 3, 1, 16, 64)
    q = randn(g, 1, 3, 2, 64)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32)
    run = lambda: B.gdn_attn_decode(q.cuda(), kb.cuda().view(F8), vb.cuda().view(F8), table.cuda(), i32([40]),
                                    k_scale=ks.cuda(), v_scale=vs.cuda(), out_dtype=F32)
    want = run()
    vb[1, 0, 39 - 32, 5] = 0x7F
    vb[1, 0, 38 - 32, 9] = 0x7F
    got = run()
    assert torch.equal(got[0, 0], want[0, 0])
    nan = torch.zeros_like(got, dtype=torch.bool)
    nan[0, 1:, :, 9] = True
    nan[0, 2, :, 5] = True
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("shared", [16, 64])
def test_decode8_shared_prefix(shared):
    run_decode([100, 70, 64, 20, 200], 4, 2, 128, 16, shared=shared)


def test_decode_weights_do_not_go_with_a_shared_prefix():
    z = torch.zeros
    kc = z(2, 1, 16, 64, dtype=BF, device="cuda")
    with pytest.raises(B.GdnError):
        B.gdn_attn_decode(z(1, 1, 64, dtype=BF, device="cuda"), kc, kc, i32([[0, 1]]), i32([17]), shared_len=16,
                          weights=z(2, 1, 16, device="cuda"))


@FORMS
def test_decode_pages_that_do_not_exist(bits, weights):
    g = torch.Generator().manual_seed(11)
    Hk, D, page = 2, 64, 16
    if bits == 8:
        kb, ks = random_cache8(g, 4, Hk, page, D, 1)
        vb, vs = random_cache8(g, 4, Hk, page, D, 1)
        kv, vv = values8(kb, ks), values8(vb, vs)
    else:
        kb, vb = randn(g, 4, Hk, page, D), randn(g, 4, Hk, page, D)
        ks = vs = None
        kv, vv = np64(kb), np64(vb)
    q = randn(g, 3, 4, D)
    table, lens = torch.tensor([[0, 9, 1], [-3, 2, 2], [3, 3, 3]], dtype=torch.int32), [40, 30, 1000]
    table[1, 2] = 1 << 30
    w = torch.rand(4, Hk, page, generator=g) if weights else None
    status = new_status()
    cuda = lambda x: None if x is None else x.cuda()
    t = F8 if bits == 8 else BF
    w_dev = cuda(w)
    out, lse = B.gdn_attn_decode(q.cuda(), cuda(kb).view(t), cuda(vb).view(t), table.cuda(), i32(lens),
                                 out_dtype=F32, return_lse=True, status=status, k_scale=cuda(ks),
                                 v_scale=cuda(vs), weights=w_dev)
    assert status.item() == 64 | 128
    ref, mag, rl = A.decode(np64(q)[:, None], kv, vv, table.numpy(), lens)
    floor = fp16_floor(np64(q)[:, None], kv, vb, vs, table, lens) if bits == 8 else 0.0
    close(out, lse, ref, mag, rl, floor)
    if weights:  # (the page that a sequence names three times gathers three times, in any order)
        want = C.decode_weights(np64(q)[:2, None], kv, table.numpy()[:2], lens[:2], w.numpy())
        assert np.abs(np64(w_dev)[:3] - want[:3]).max() < 1e-4


def test_decode8_cache_past_32_bit_offsets():
    """A cache of more than 2^32 bytes, the sequence's pages at its end."""
    Hk, page, D = 8, 256, 128
    n_pages = (1 << 32) // (Hk * page * D) + 4
    g = torch.Generator().manual_seed(12)
    b, s = random_cache8(g, 4, Hk, page, D, 1)
    kc = torch.zeros(n_pages, Hk, page, D, dtype=torch.uint8, device="cuda")
    ks = torch.zeros(n_pages, Hk, page // 16, device="cuda")
    kc[-4:], ks[-4:] = b.cuda(), s.cuda()
    table = torch.tensor([[n_pages - 1, n_pages - 3]], dtype=torch.int32)
    q = randn(g, 1, 8, D)
    w = torch.zeros(n_pages, Hk, page, device="cuda")
    out, lse = B.gdn_attn_decode(q.cuda(), kc.view(F8), kc.view(F8), table.cuda(), i32([400]), out_dtype=F32,
                                 return_lse=True, k_scale=ks, v_scale=ks, weights=w)
    v = values8(b, s)
    t = table.numpy() - (n_pages - 4)
    floor = fp16_floor(np64(q)[:, None], v, b, s, torch.from_numpy(t), [400])
    close(out, lse, *A.decode(np64(q)[:, None], v, v, t, [400]), floor)
    want = C.decode_weights(np64(q)[:, None], v, t, [400], np.zeros((4, Hk, page)))
    assert np.abs(np64(w[-4:]) - want).max() < 1e-4 and w[:-4].abs().max() == 0
    x = randn(g, 16, Hk, D)
    B.gdn_attn_append8(x.cuda(), x.cuda(), kc.view(F8), kc.view(F8), ks, ks, table.cuda(), kv_lens=i32([416]))
    want, ws = C.append8(np64(x), b.numpy(), s.numpy(), t, [416])
    assert C.same_bytes(as_bytes(kc[-4:]), want).all() and np.array_equal(ks[-4:].cpu().numpy(), ws)
    new = i32([[n_pages - 2]])
    lens, kept = B.gdn_attn_evict(kc.view(F8), kc.view(F8), w, table.cuda(), i32([416]), new, 200, 16, ks, ks)
    dst, wl, wk = C.evict(want, want, np64(w[-4:]), t, [416], np.array([[2]]), 200, 16, ws, ws)
    assert np.array_equal(kept.cpu().numpy(), wk) and C.same_bytes(as_bytes(kc[-4:]), dst[0]).all()


# ---------------------------------------------------------------- a prompt's weights
def run_prompt(lens, H, Hk, D, page=16, window=0, seed=0, lead=0, tail=0, mul=1.0, scale=None, slack=0.0):
    g = torch.Generator().manual_seed(seed)
    T = lead + sum(lens) + tail
    q, k = randn(g, T, H, D, mul=mul), randn(g, T, Hk, D)
    cu = torch.tensor([lead] + lens).cumsum(0).to(torch.int32)
    table, n_pages, _ = pages_for(g, [-(-n // page) for n in lens], 1)
    w = torch.rand(n_pages, Hk, page, generator=g)
    lse = A.prefill(np64(q), np64(k), np64(k), cu.numpy(), scale)[2]
    lse = torch.from_numpy(np.where(np.isfinite(lse), lse, 0.0)).float()
    w_dev, status = w.cuda(), new_status()
    B.gdn_attn_prefill_weights(q.cuda(), k.cuda(), lse.cuda(), w_dev, table.cuda(), cu_seqlens=cu.cuda(),
                               window=window, scale=scale, status=status)
    assert status.item() == 0
    want = C.prefill_weights(np64(q), np64(k), np64(lse), w.numpy(), table.numpy(), cu.numpy(), window, scale)
    rel = weight_slack(q, np64(k), D, scale or D ** -0.5) + slack
    got = np64(w_dev)
    bad = ~(np.abs(got - want) <= rel * want + 1e-9)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], rel)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("L", [1, 2, 31, 63, 64, 65, 127, 128, 129, 255, 257, 400])
def test_prompt_lengths(L, D):
    run_prompt([L], 2, 1, D, seed=L)


@pytest.mark.parametrize("H, Hk", [(1, 1), (3, 3), (3, 1), (5, 1), (6, 2), (7, 1), (16, 2), (24, 2), (33, 1), (64, 1)])
def test_prompt_groups(H, Hk):
    run_prompt([70, 1, 150], H, Hk, 128, seed=H)


@pytest.mark.parametrize("lens", [[0, 5, 0, 130, 1, 0], [300, 1, 1, 64], [128, 128], [1] * 70, [3, 250, 17, 129, 66]])
@pytest.mark.parametrize("D", [64, 128])
def test_prompt_packed(lens, D):
    run_prompt(lens, 4, 2, D, seed=len(lens), lead=3, tail=9, page=32)


@pytest.mark.parametrize("window", [1, 2, 17, 64, 127, 128, 129, 200, 5000])
def test_prompt_windows(window):
    run_prompt([300, 1, 129, 40], 4, 2, 128, window=window)
    run_prompt([257], 3, 1, 64, window=window)


@pytest.mark.parametrize("mul", [0.01, 4.0, 8.0])
def test_prompt_score_ranges(mul):
    run_prompt([385], 2, 1, 128, mul=mul)


def test_prompt_scale_and_pages():
    run_prompt([200], 4, 1, 128, scale=0.3)
    run_prompt([300, 20], 4, 1, 64, page=256)


@pytest.mark.parametrize("scale", [2.0 ** -100, 1e-6, 20.0])
def test_prompt_scales_far_from_the_usual(scale):
    """lse / scale is formed: 1 / scale and the quotient rounded (a half step of 2^-24 each), its three
    parts in bf16 (2^-25), the sum of it and the product (2^-23, as it may be cut), scale * log2(e)
    and that times the sum (2^-24 each): 6.5 * 2^-24 |lse| at most, |lse| <= log(150) + 0.01 where
    scores are nothing beside it."""
    run_prompt([150, 20], 4, 2, 64, scale=scale, slack=6.5 * 2.0 ** -24 * 5.03)


def test_prompt_many_sequences():
    run_prompt([1 + 13 * i % 9 if i % 5 else 0 for i in range(1100)] + [140, 0, 3], 2, 1, 64)


def test_prompt_longer():
    run_prompt([1500], 2, 1, 128)


def test_prompt_keys_of_other_rows_have_no_influence():
    """Rows before a key, padding, and what the window leaves out: NaN there changes nothing."""
    g = torch.Generator().manual_seed(6)
    T, H, Hk, D = 200, 2, 1, 64
    q, k = randn(g, T, H, D), randn(g, T, Hk, D)
    lse = torch.rand(T, H, generator=g) + 4
    cu, table = i32([3, 150]), i32([list(range(10))])
    run = lambda: B.gdn_attn_prefill_weights(q.cuda(), k.cuda(), lse.cuda(), w, table, cu_seqlens=cu, window=20)
    w = torch.zeros(10, Hk, 16, device="cuda")
    run()
    want, w = w, torch.zeros_like(w)
    q[:130] = float("nan")
    lse[:130] = float("nan")
    q[150:], k[:3], k[150:], lse[150:] = float("nan"), float("inf"), float("nan"), float("-inf")
    run()
    assert torch.equal(w, want) and w.isfinite().all()
    # a key that some rows of the window do not see: its NaN is its own
    k[149] = float("nan")
    run()
    w = w.transpose(0, 1).reshape(Hk, -1)
    assert w[0, 146].isnan() and torch.equal(w[0, :146], want.transpose(0, 1).reshape(Hk, -1)[0, :146])


def test_prompt_places_that_do_not_exist():
    g = torch.Generator().manual_seed(7)
    T, H, Hk, D = 100, 2, 1, 64
    q, k = randn(g, T, H, D), randn(g, T, Hk, D)
    lse = np.where(True, A.prefill(np64(q), np64(k), np64(k), [0, 60, 100])[2], 0)
    table = i32([[0, 9, 1], [-1, 2, 2]])  # the first sequence is longer than its row
    w = torch.full((4, Hk, 16), 7.0, device="cuda")
    status = new_status()
    B.gdn_attn_prefill_weights(q.cuda(), k.cuda(), torch.from_numpy(lse).float().cuda(), w, table,
                               cu_seqlens=i32([0, 60, 100]), status=status)
    assert status.item() == 64 | 128
    want = C.prefill_weights(np64(q), np64(k), lse, np.full((4, Hk, 16), 7.0), table.cpu().numpy(), [0, 60, 100])
    got = np64(w)
    assert np.abs(got[[0, 1, 3]] - want[[0, 1, 3]]).max() < 1e-3  # (page 2 is named twice)


def test_prompt_malformed_cu_seqlens():
    g = torch.Generator().manual_seed(8)
    T, H, Hk, D = 150, 2, 1, 64
    q, k = randn(g, T, H, D), randn(g, T, Hk, D)
    for cu in ([0, 100, 50, 150], [-5, 40, 150], [0, 90, 1000], [140, 20, 10]):
        N = len(cu) - 1
        sane = A.sane_bounds(cu, T)
        lse = A.prefill(np64(q), np64(k), np64(k), cu)[2]
        lse = torch.from_numpy(np.where(np.isfinite(lse), lse, 0.0)).float()
        table = torch.arange(10 * N, dtype=torch.int32).reshape(N, 10)
        w, status = torch.zeros(10 * N, Hk, 16, device="cuda"), new_status()
        B.gdn_attn_prefill_weights(q.cuda(), k.cuda(), lse.cuda(), w, table.cuda(), cu_seqlens=i32(cu), status=status)
        assert status.item() == 1
        want = C.prefill_weights(np64(q), np64(k), np64(lse), np.zeros((10 * N, Hk, 16)), table.numpy(), sane)
        assert np.abs(np64(w) - want).max() < 1e-3


# ---------------------------------------------------------------- evict
def run_evict(lens, Hk, D, page, keep, recent, bits=16, seed=0, change=None, alias=False, power=True):
    g = torch.Generator().manual_seed(seed)
    N = len(lens)
    fresh = [-(-min(max(n, 0), keep) // page) for n in lens]
    table, n_pages, spare = pages_for(g, [-(-max(n, 0) // page) for n in lens], sum(fresh) + 1)
    new = torch.full((N, -(-keep // page)), -1, dtype=torch.int32)
    for n, c in enumerate(fresh):
        for i in range(c):
            new[n, i] = spare.pop()
    w = torch.exp(4 * torch.randn(n_pages, Hk, page, generator=g))
    w[torch.rand(w.shape, generator=g) < 0.3] = 0.0
    w[torch.rand(w.shape, generator=g) < 0.2] = 1.5
    if change:
        w = change(w)
    ks = vs = None
    if bits == 8:
        kb, ks = random_cache8(g, n_pages, Hk, page, D, 4, power)
        vb, vs = random_cache8(g, n_pages, Hk, page, D, 4, power)
        ks[0] = 0.0
    else:
        kb, vb = randn(g, n_pages, Hk, page, D), randn(g, n_pages, Hk, page, D)
    raw = (lambda x: x.numpy()) if bits == 8 else (lambda x: x.view(torch.int16).numpy())
    dst, want_lens, want_kept = C.evict(raw(kb), raw(vb), w.numpy(), table.numpy(), lens, new.numpy(), keep, recent,
                                        None if ks is None else ks.numpy(), None if vs is None else vs.numpy())
    cuda = lambda x: None if x is None else x.cuda()
    t = F8 if bits == 8 else BF
    k_dev, v_dev, w_dev, ks_dev, vs_dev = (cuda(x) for x in (kb, vb, w, ks, vs))
    status, kv = new_status(), i32(lens)
    got_lens, kept = B.gdn_attn_evict(k_dev.view(t), v_dev.view(t), w_dev, table.cuda(), kv, new.cuda(), keep, recent,
                                      k_scale=ks_dev, v_scale=vs_dev, new_lens=kv if alias else None, status=status)
    assert status.item() == 0
    assert np.array_equal(got_lens.cpu().numpy(), want_lens)
    assert np.array_equal(kept.cpu().numpy(), want_kept)
    if alias:
        assert got_lens.data_ptr() == kv.data_ptr()
    back = lambda x: raw(x.cpu())
    if bits == 8:
        for x, y in ((k_dev, dst[0]), (v_dev, dst[1])):
            a, b = C.VALUES[back(x)], C.VALUES[y]
            near = np.abs(a - b) <= (0.0 if power else 2.0 ** -3 * np.abs(b) + 2.0 ** -9)
            assert (near | (np.isnan(a) & np.isnan(b))).all()
        assert np.array_equal(ks_dev.cpu().numpy(), dst[3]) and np.array_equal(vs_dev.cpu().numpy(), dst[4])
    else:
        assert np.array_equal(back(k_dev), dst[0]) and np.array_equal(back(v_dev), dst[1])
    assert np.array_equal(w_dev.cpu().numpy(), dst[2], equal_nan=True)


BITS = pytest.mark.parametrize("bits", [8, 16])


@BITS
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_evict_pages(page, D, bits):
    run_evict([3 * page + 5, page, 1, 0, 400], 2, D, page, 100, 10, bits, seed=page)


@BITS
@pytest.mark.parametrize("keep, recent", [(1, 0), (1, 1), (2, 1), (15, 15), (16, 0), (17, 3), (33, 32), (64, 0),
                                          (199, 20), (200, 20), (300, 0)])
def test_evict_budgets(keep, recent, bits):
    run_evict([200, 201, 16, 17, 600], 3, 64, 16, keep, recent, bits, seed=keep)


@BITS
def test_evict_many_and_long(bits):
    run_evict([1 + 97 * i % 300 for i in range(60)], 4, 64, 32, 70, 8, bits)
    run_evict([9000, 5, 4097], 2, 64, 64, 1000, 100, bits)


@pytest.mark.parametrize("longest", [2048, 4096, 8192, 16384, 32768, 40000])
def test_evict_row_lengths(longest):
    """Each size of the selection, full and nearly empty; weights of many equal values."""
    run_evict([longest, 9, longest - 1, longest // 2 + 3], 1, 64, 256, longest // 3, 17, seed=longest)
    run_evict([longest - 5], 2, 64, 16, 50, 0, 8, change=lambda w: (w * 3).round())


@pytest.mark.parametrize("longest", [2048, 4096, 8192, 16384, 32768])
def test_evict_rows_that_stay_nearly_whole(longest):
    """Every lane of a warp keeps all of its tokens, in one go or up to the first equal ones."""
    run_evict([longest, longest - 1], 1, 64, 256, longest - 3, 1, seed=longest)
    run_evict([longest], 1, 64, 256, longest - 40, 0, 8, change=torch.ones_like)


@pytest.mark.parametrize("what", ["equal", "zeros", "negative", "nan", "inf", "close", "denormal"])
def test_evict_choices(what):
    def change(w):
        g = torch.Generator().manual_seed(1)
        if what == "equal":
            return torch.full_like(w, 2.5)
        if what == "zeros":
            return torch.where(torch.rand(w.shape, generator=g) < 0.5, 0.0, -0.0)
        if what == "negative":
            return torch.randn(w.shape, generator=g).round(decimals=1)
        if what == "nan":
            return torch.where(torch.rand(w.shape, generator=g) < 0.2, float("nan"), w)
        if what == "inf":
            return torch.where(torch.rand(w.shape, generator=g) < 0.2, float("inf"), -w)
        if what == "close":  # differ in the last bits only
            return (0x3F800000 + torch.randint(0, 40, w.shape, generator=g)).to(torch.int32).view(F32)
        return torch.randint(0, 50, w.shape, generator=g).to(torch.int32).view(F32)
    run_evict([700, 100, 513], 2, 64, 16, 90, 7, change=change)


@BITS
def test_evict_in_place_lengths(bits):
    run_evict([200, 20, 90], 2, 128, 32, 50, 5, bits, alias=True)


def test_evict_scales_that_are_no_powers_of_two():
    run_evict([200, 20, 90], 2, 128, 32, 50, 5, 8, power=False)


@BITS
def test_evict_pages_that_do_not_exist(bits):
    g = torch.Generator().manual_seed(2)
    Hk, D, page = 2, 64, 16
    table = torch.tensor([[0, 9, 1], [-1, 2, 3]], dtype=torch.int32)
    new = torch.tensor([[5, 11], [-7, 6]], dtype=torch.int32)
    lens, keep, recent = [45, 10000], 20, 4
    w = torch.rand(8, Hk, page, generator=g)
    if bits == 8:
        kb, ks = random_cache8(g, 8, Hk, page, D)
        raw = lambda x: x.numpy()
    else:
        kb, ks = randn(g, 8, Hk, page, D), None
        raw = lambda x: x.view(torch.int16).numpy()
    k_dev, v_dev, w_dev = kb.cuda(), kb.cuda(), w.cuda()
    s_dev = [None if ks is None else ks.cuda() for _ in range(2)]
    status = new_status()
    got, kept = B.gdn_attn_evict(k_dev.view(F8 if bits == 8 else BF), v_dev.view(F8 if bits == 8 else BF), w_dev,
                                 table.cuda(), i32(lens), new.cuda(), keep, recent, k_scale=s_dev[0], v_scale=s_dev[1],
                                 status=status)
    assert status.item() == 64 | 128
    s = None if ks is None else ks.numpy()
    dst, want_lens, want_kept = C.evict(raw(kb), raw(kb), w.numpy(), table.numpy(), lens, new.numpy(), keep, recent, s, s)
    assert np.array_equal(got.cpu().numpy(), want_lens) and np.array_equal(kept.cpu().numpy(), want_kept)
    assert np.array_equal(w_dev.cpu().numpy(), dst[2])
    for x in (k_dev, v_dev):
        assert (C.same_bytes(raw(x.cpu()), dst[0]).all() if bits == 8 else np.array_equal(raw(x.cpu()), dst[0]))


# ---------------------------------------------------------------- the front end's positions
def run_axes(T, H, Hk, D, rot, inter, axes, n_axes=3, x_dtype=BF, out_dtype=None, cache=True, lens=None, pasts=None,
             norm=True, seed=0, positions=None, max_pos=500, want_status=0):
    g = torch.Generator().manual_seed(seed)
    x = randn(g, T, (H + 2 * Hk) * D, dtype=x_dtype, mul=2.0)
    qw, kw = (randn(g, D, dtype=F32, mul=0.2) + 1 for _ in range(2)) if norm else (None, None)
    rope = rope_table(max_pos, rot, device="cpu")
    pos = torch.randint(0, max_pos, (n_axes, T), generator=g, dtype=torch.int32) if positions is None else positions
    lens, pasts = lens or [T], pasts or [0] * len(lens or [T])
    ends = [a + b for a, b in zip(lens, pasts)]
    table, n_pages, _ = pages_for(g, [-(-e // 16) for e in ends], 1)
    out_dtype = out_dtype or x_dtype
    kc, vc = (randn(g, n_pages, Hk, 16, D, dtype=out_dtype) for _ in range(2))
    dev = lambda t: None if t is None else t.cuda()
    kd, vd, status = dev(kc), dev(vc), new_status()
    more = dict(page_table=table.cuda(), k_cache=kd, v_cache=vd, kv_lens=i32(ends)) if cache else {}
    cu = np.cumsum([0] + lens)
    q, k, v = B.gdn_attn_front(x.cuda(), H, Hk, D, dev(qw), dev(kw), rope=rope.cuda(), interleaved=inter,
                               cu_seqlens=i32(cu.tolist()), out_dtype=out_dtype, status=status, positions=pos.cuda(),
                               rope_axes=dev(axes), **more)
    assert status.item() == want_status
    wq, wk = C.front_axes(np64(x), H, Hk, D, None if qw is None else np64(qw), None if kw is None else np64(kw), 1e-6,
                          np64(rope), inter, pos.numpy(), None if axes is None else axes.numpy())
    wv = np64(x).reshape(T, -1, D)[:, H + Hk:]
    for got, want in ((q, wq), (k, wk), (v, wv)):
        size = np.abs(want).max(-1, keepdims=True)
        tol = 2e-6 * size + (2.0 ** -8 * np.abs(want) if out_dtype == BF else 0)
        assert (np.abs(np64(got) - want) <= tol + 1e-30).all()
    if cache:
        for got, was, dense in ((kd, kc, k), (vd, vc, v)):
            want = was.clone()
            for n in range(len(lens)):
                for i in range(lens[n]):
                    at = pasts[n] + i
                    want[int(table[n, at // 16]), :, at % 16] = dense[cu[n] + i].cpu()
            assert torch.equal(got.cpu(), want)


def axes_of(kind, half, n):
    i = torch.arange(half)
    return {"cyclic": i % n, "sections": i * n // half, "none": None}[kind].to(torch.uint8) if kind != "none" else None


@pytest.mark.parametrize("kind", ["cyclic", "sections", "none"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D, rot", [(64, 64), (64, 16), (128, 128), (128, 32), (128, 96)])
def test_axes_rotary(D, rot, inter, kind):
    run_axes(9, 4, 2, D, rot, inter, axes_of(kind, rot // 2, 3))


@pytest.mark.parametrize("n_axes", [1, 2, 4, 8])
def test_axes_counts(n_axes):
    run_axes(20, 2, 1, 128, 64, False, axes_of("cyclic", 32, n_axes), n_axes=n_axes)


@pytest.mark.parametrize("x_dtype, out_dtype", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("D", [64, 128])
def test_axes_types(D, x_dtype, out_dtype):
    run_axes(33, 2, 2, D, 32, True, axes_of("cyclic", 16, 3), x_dtype=x_dtype, out_dtype=out_dtype)


@pytest.mark.parametrize("norm, cache", [(False, False), (True, False), (False, True)])
def test_axes_parts(norm, cache):
    run_axes(12, 4, 1, 64, 64, False, axes_of("sections", 32, 2), n_axes=2, norm=norm, cache=cache)


def test_axes_sequences_keep_their_places():
    """The cache's places come from the lengths, whatever the positions are."""
    run_axes(60, 4, 2, 128, 64, False, axes_of("cyclic", 32, 3), lens=[1, 40, 0, 19], pasts=[17, 3, 5, 0])
    run_axes(64, 2, 1, 64, 32, False, axes_of("cyclic", 16, 3), lens=[1] * 64, pasts=list(range(64)))


def test_axes_many_rows():
    run_axes(2500, 8, 2, 64, 32, True, axes_of("cyclic", 16, 3))


def test_axes_outside_the_table():
    pos = torch.tensor([[-1, 3, 500], [1 << 30, 4, -(1 << 31)], [2, 499, 0]], dtype=torch.int32)
    run_axes(3, 2, 1, 64, 32, False, axes_of("cyclic", 16, 3), positions=pos, want_status=128)
    axes = axes_of("cyclic", 16, 3)
    axes[3], axes[7] = 3, 255
    run_axes(3, 2, 1, 64, 32, False, axes, want_status=128)


def test_axes_all_the_places_are_the_plain_call():
    g = torch.Generator().manual_seed(4)
    T, H, Hk, D = 50, 4, 2, 128
    x = randn(g, T, (H + 2 * Hk) * D).cuda()
    rope = rope_table(100, 64)
    lens = i32([70])
    pos = torch.arange(20, 70, dtype=torch.int32, device="cuda").repeat(3, 1)
    plain = B.gdn_attn_front(x, H, Hk, D, rope=rope, kv_lens=lens)
    axes = B.gdn_attn_front(x, H, Hk, D, rope=rope, kv_lens=lens, positions=pos,
                            rope_axes=axes_of("cyclic", 32, 3).cuda())
    assert all(torch.equal(a, b) for a, b in zip(plain, axes))


# ---------------------------------------------------------------- graphs, streams, bounds
def all_calls(seed=0, N=5, Hk=2, G=3, D=64, page=16):
    """Each operator as a call that writes into tensors of its own: (run, outputs, restore)."""
    g = torch.Generator().manual_seed(seed)
    H = Hk * G
    lens = [50, 1, 90, 33, 200][:N]
    table, n_pages, spare = pages_for(g, [-(-n // page) for n in lens], 20)
    new = torch.tensor(spare[:N * 2], dtype=torch.int32).reshape(N, 2).cuda()
    kb, ks = random_cache8(g, n_pages, Hk, page, D, 1)
    vb, vs = random_cache8(g, n_pages, Hk, page, D, 1)
    k8, v8, ks, vs = kb.cuda().view(F8), vb.cuda().view(F8), ks.cuda(), vs.cuda()
    k16, v16 = randn(g, n_pages, Hk, page, D).cuda(), randn(g, n_pages, Hk, page, D).cuda()
    w = torch.rand(n_pages, Hk, page, generator=g).cuda()
    q = randn(g, N, H, D).cuda()
    T = sum(lens)
    kv, cu = i32(lens), i32(np.cumsum([0] + lens).tolist())
    table = table.cuda()
    xk, xv = randn(g, T, Hk, D).cuda(), randn(g, T, Hk, D).cuda()
    xq, lse = randn(g, T, H, D).cuda(), (torch.rand(T, H, generator=g) + 4).cuda()
    out = torch.zeros(N, H, D, dtype=BF, device="cuda")
    desc = B.make_attn_desc(N, N, H, Hk, D, page_size=page, n_pages=n_pages, max_pages=table.shape[1])
    work = torch.zeros(B.gdn_attn_decode_cache_workspace_size(desc, True), dtype=torch.uint8, device="cuda")
    pdesc = B.make_attn_desc(T, N, H, Hk, D, page_size=page, n_pages=n_pages, max_pages=table.shape[1])
    pwork = torch.zeros(B.gdn_attn_prefill_weights_workspace_size(pdesc), dtype=torch.uint8, device="cuda")
    new_lens, kept = torch.zeros(N, dtype=torch.int32, device="cuda"), torch.zeros(N, Hk, 20, dtype=torch.int32, device="cuda")
    xa = randn(g, T, (H + 2 * Hk) * D).cuda()
    rope, pos = rope_table(300, 32), torch.randint(0, 300, (3, T), generator=g, dtype=torch.int32).cuda()
    fq = torch.zeros(T, H, D, dtype=BF, device="cuda")
    state = [k8, v8, ks, vs, k16, v16, w, out, new_lens, kept, fq]
    keep = [x.clone() for x in state]

    def restore():
        for x, y in zip(state, keep):
            x.copy_(y)
    calls = dict(
        append8=lambda s=None: B.gdn_attn_append8(xk, xv, k8, v8, ks, vs, table, kv, cu, stream=s),
        decode8=lambda s=None: B.gdn_attn_decode(q, k8, v8, table, kv, k_scale=ks, v_scale=vs, out=out, workspace=work, stream=s),
        weights8=lambda s=None: B.gdn_attn_decode(q, k8, v8, table, kv, k_scale=ks, v_scale=vs, weights=w, out=out, workspace=work, stream=s),
        weights16=lambda s=None: B.gdn_attn_decode(q, k16, v16, table, kv, weights=w, out=out, workspace=work, stream=s),
        prompt=lambda s=None: B.gdn_attn_prefill_weights(xq, xk, lse, w, table, cu, workspace=pwork, stream=s),
        evict8=lambda s=None: B.gdn_attn_evict(k8, v8, w, table, kv, new, 20, 3, ks, vs, new_lens, kept, stream=s),
        evict16=lambda s=None: B.gdn_attn_evict(k16, v16, w, table, kv, new, 20, 3, None, None, new_lens, kept, stream=s),
        front=lambda s=None: B.gdn_attn_front(xa, H, Hk, D, rope=rope, cu_seqlens=cu, kv_lens=kv, page_table=table, k_cache=k16,
                                              v_cache=v16, output_kv=False, q=fq, positions=pos, stream=s))
    return calls, state, restore


CALLS = ["append8", "decode8", "weights8", "weights16", "prompt", "evict8", "evict16", "front"]


def snapshot(state):
    return [x.view(torch.uint8).clone() for x in state]


@pytest.mark.parametrize("name", CALLS)
def test_repeatable_other_stream_and_graph(name):
    calls, state, restore = all_calls()
    run = calls[name]
    run()
    torch.cuda.synchronize()
    want = snapshot(state)
    restore()
    run()
    assert all(torch.equal(a, b) for a, b in zip(snapshot(state), want))
    restore()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(snapshot(state), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(2):
        restore()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(snapshot(state), want))


@pytest.mark.parametrize("name", ["decode8", "weights8", "prompt", "evict16"])
def test_memory_that_the_call_allocates(name):
    """Without outputs and workspace given, on a stream of its own."""
    calls, state, restore = all_calls(seed=1)
    calls[name]()
    want = snapshot(state)
    restore()
    g = torch.Generator().manual_seed(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = calls[name].__closure__
    env = {n: x.cell_contents for n, x in zip(calls[name].__code__.co_freevars, c)}
    if name == "prompt":
        B.gdn_attn_prefill_weights(env["xq"], env["xk"], env["lse"], env["w"], env["table"], env["cu"], stream=side)
    elif name == "evict16":
        got = B.gdn_attn_evict(env["k16"], env["v16"], env["w"], env["table"], env["kv"], env["new"], 20, 3, stream=side)
    else:
        got = B.gdn_attn_decode(env["q"], env["k8"], env["v8"], env["table"], env["kv"], k_scale=env["ks"],
                                v_scale=env["vs"], weights=env.get("w"), stream=side)
    torch.cuda.current_stream().wait_stream(side)
    if name == "evict16":
        env["new_lens"].copy_(got[0]), env["kept"].copy_(got[1])
    elif name != "prompt":
        env["out"].copy_(got)
    assert all(torch.equal(a, b) for a, b in zip(snapshot(state), want))
    del g


def test_outputs_and_workspaces_stay_in_their_bounds():
    """Everything in one buffer with guards between, checked after each call."""
    g = torch.Generator().manual_seed(3)
    N, Hk, G, D, page = 4, 2, 5, 128, 32
    H, lens = Hk * G, [100, 1, 65, 300]
    table, n_pages, spare = pages_for(g, [-(-n // page) for n in lens], 12)
    T = sum(lens)
    desc = B.make_attn_desc(N, N, H, Hk, D, page_size=page, n_pages=n_pages, max_pages=table.shape[1])
    pdesc = B.make_attn_desc(T, N, H, Hk, D, page_size=page, n_pages=n_pages, max_pages=table.shape[1])
    sizes = dict(k8=(n_pages, Hk, page, D, F8), v8=(n_pages, Hk, page, D, F8), ks=(n_pages, Hk, page // 16, F32),
                 vs=(n_pages, Hk, page // 16, F32), w=(n_pages, Hk, page, F32), out=(N, H, D, BF), lse=(N, H, F32),
                 work=(B.gdn_attn_decode_cache_workspace_size(desc, True), torch.uint8),
                 pwork=(B.gdn_attn_prefill_weights_workspace_size(pdesc), torch.uint8),
                 new_lens=(N, torch.int32), kept=(N, Hk, 40, torch.int32))
    at, views = 4096, {}
    spans = []
    for name, (*shape, dtype) in sizes.items():
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        spans.append((name, at, n, shape, dtype))
        at = (at + n + 255) // 256 * 256 + 4096
    buf = torch.full((at,), 0x5A, dtype=torch.uint8, device="cuda")
    used = torch.zeros(at, dtype=torch.bool, device="cuda")
    for name, b, n, shape, dtype in spans:
        views[name] = buf[b:b + n].view(dtype).view(shape)
        used[b:b + n] = True
    kb, s = random_cache8(g, n_pages, Hk, page, D, 1)
    views["k8"].view(torch.uint8).copy_(kb), views["v8"].view(torch.uint8).copy_(kb)
    views["ks"].copy_(s), views["vs"].copy_(s), views["w"].fill_(1.0)
    v, kv, cu, table = views, i32(lens), i32(np.cumsum([0] + lens).tolist()), table.cuda()
    new = torch.tensor(spare[:2 * N], dtype=torch.int32).reshape(N, 2).cuda()
    xk, xq = randn(g, T, Hk, D).cuda(), randn(g, T, H, D).cuda()
    lse = (torch.rand(T, H, generator=g) + 4).cuda()
    B.gdn_attn_append8(xk, xk, v["k8"], v["v8"], v["ks"], v["vs"], table, kv, cu)
    B.gdn_attn_decode(randn(g, N, H, D).cuda(), v["k8"], v["v8"], table, kv, k_scale=v["ks"], v_scale=v["vs"],
                      weights=v["w"], out=v["out"], return_lse=True, lse=v["lse"], workspace=v["work"])
    B.gdn_attn_prefill_weights(xq, xk, lse, v["w"], table, cu, workspace=v["pwork"])
    B.gdn_attn_evict(v["k8"], v["v8"], v["w"], table, kv, new, 40, 4, v["ks"], v["vs"], v["new_lens"], v["kept"])
    assert (buf[~used] == 0x5A).all()


def test_two_graphs_with_workspaces_of_their_own():
    """Replayed in turn and at once on two streams."""
    sets = [all_calls(seed=s) for s in (5, 6)]
    wants, graphs = [], []
    for calls, state, restore in sets:
        calls["weights8"]()
        wants.append(snapshot(state))
        restore()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            calls["weights8"]()
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for calls, state, restore in sets:
            restore()
        torch.cuda.synchronize()
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for want, (calls, state, restore) in zip(wants, sets):
            assert all(torch.equal(a, b) for a, b in zip(snapshot(state), want))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("call", ["decode8", "decode8_rows", "decode8_weights", "prompt"])
@pytest.mark.parametrize("item", [0, 1, 2])
def test_a_wait_that_runs_out_is_reported_and_leaves_the_next_call_right(call, D, item):
    """The testing hook has a wait before a CTA's first, second or third work item run out: the call
    returns with GDN_DEV_TIMEOUT, and with the hook off the same call on the same buffers gives
    its results again."""
    g = torch.Generator().manual_seed(52)
    status = new_status()
    if call == "prompt":
        q, k = (randn(g, 5000, h, D).cuda() for h in (8, 2))
        cu = i32([0, 2000, 2001, 5000])
        table = torch.arange(3 * 24, dtype=torch.int32, device="cuda").reshape(3, 24)
        lse = torch.full((5000, 8), 6.0, device="cuda")
        size = B.gdn_attn_prefill_weights_workspace_size(B.make_attn_desc(
            5000, 3, 8, 2, D, page_size=128, n_pages=72, max_pages=24))
        work = torch.empty(size, dtype=torch.uint8, device="cuda")

        def run():
            w = torch.zeros(72, 2, 128, device="cuda")
            B.gdn_attn_prefill_weights(q, k, lse, w, table, cu, workspace=work, status=status)
            return (w,)
    else:
        N, Hk, nq = 200, 4, 5 if call == "decode8_rows" else 1
        kb, ks = random_cache8(g, N * 8, Hk, 128, D)
        vb, vs = random_cache8(g, N * 8, Hk, 128, D)
        kb, vb, ks, vs = kb.cuda().view(F8), vb.cuda().view(F8), ks.cuda(), vs.cuda()
        table = torch.randperm(N * 8, generator=g).to(torch.int32).reshape(N, 8).cuda()
        kv = torch.randint(600, 1025, (N,), generator=g).to(torch.int32).cuda()
        q = randn(g, N, nq, 5 * Hk, D).cuda()
        kinds = dict(with_weights=call == "decode8_weights")
        size = B.gdn_attn_decode_cache_workspace_size(B.make_attn_desc(
            N * nq, N, 5 * Hk, Hk, D, page_size=128, n_pages=N * 8, max_pages=8), **kinds)
        work = torch.empty(size, dtype=torch.uint8, device="cuda")

        def run():
            w = torch.zeros(N * 8, Hk, 128, device="cuda") if call == "decode8_weights" else None
            out = B.gdn_attn_decode(q, kb, vb, table, kv, k_scale=ks, v_scale=vs, weights=w, workspace=work,
                                    status=status)
            return (out,) if w is None else (out, w)
    want = run()
    assert status.item() == 0
    try:
        B.gdn_test_attn_timeout(256, item)
        run()
        assert status.item() & 8
    finally:
        B.gdn_test_attn_timeout(0)
    got = run()
    assert status.item() == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_tokens():
    e = lambda *s, t=BF: torch.empty(*s, dtype=t, device="cuda")
    k8, ks = e(2, 1, 16, 64, t=F8), e(2, 1, 1, t=F32)
    st = new_status()
    B.gdn_attn_append8(e(0, 1, 64), e(0, 1, 64), k8, k8, ks, ks, i32([[0]]), status=st)
    assert st.item() == 0
    st = new_status()
    B.gdn_attn_prefill_weights(e(0, 2, 64), e(0, 1, 64), e(0, 2, t=F32), e(2, 1, 16, t=F32), i32([[0]]), status=st)
    assert st.item() == 0


# ---------------------------------------------------------------- together
@BITS
def test_a_conversation(bits):
    """A prompt with an image, its weights, a cut, and steps after it with positions that go on from
    the prompt's, against the oracle from the calls' own bf16 tensors."""
    g = torch.Generator().manual_seed(21)
    H, Hk, D, page, rot, keep, recent = 4, 2, 64, 16, 32, 48, 16
    N, lens = 2, [130, 40]
    T = sum(lens)
    cu = np.cumsum([0] + lens)
    axes = axes_of("sections", rot // 2, 3)
    rope = rope_table(400, rot)
    pos = torch.cat([torch.arange(n, dtype=torch.int32).repeat(3, 1) for n in lens], 1)
    pos[1, 20:80] = 20 + torch.arange(60, dtype=torch.int32) // 10
    pos[2, 20:80] = 20 + torch.arange(60, dtype=torch.int32) % 10
    table, n_pages, spare = pages_for(g, [10, 4], 10)
    new = torch.tensor(spare[:8], dtype=torch.int32).reshape(N, 4)
    x = randn(g, T, (H + 2 * Hk) * D, mul=2.0)
    one = torch.ones(D, device="cuda")
    caches = {}
    if bits == 8:
        z8, s8 = torch.zeros(n_pages, Hk, page, D, dtype=torch.uint8), torch.zeros(n_pages, Hk, 1)
        caches = dict(k_cache=z8.cuda().view(F8), v_cache=z8.cuda().view(F8))
        scales = dict(k_scale=s8.cuda(), v_scale=s8.cuda())
    else:
        z = torch.zeros(n_pages, Hk, page, D, dtype=BF)
        caches = dict(k_cache=z.cuda(), v_cache=z.cuda())
        scales = {}
    w = torch.full((n_pages, Hk, page), float("nan"), device="cuda")
    table_d, cu_d = table.cuda(), i32(cu.tolist())

    def front(x, positions, kv, cu, table):
        more = dict(page_table=table, kv_lens=kv, **caches) if bits == 16 else {}
        q, k, v = B.gdn_attn_front(x.cuda(), H, Hk, D, one, one, rope=rope, cu_seqlens=cu, positions=positions.cuda(),
                                   rope_axes=axes.cuda(), **more)
        if bits == 8:
            B.gdn_attn_append8(k, v, caches["k_cache"], caches["v_cache"], scales["k_scale"], scales["v_scale"], table, kv, cu)
        return q, k, v

    kv = i32(lens)
    q, k, v = front(x, pos, kv, cu_d, table_d)
    out, lse = B.gdn_attn_prefill(q, k, v, cu_d, return_lse=True)
    ref, mag, rl, _ = A.prefill(np64(q), np64(k), np64(v), cu)
    assert (np.abs(np64(out) - ref) <= REL * mag + 2.0 ** -8 * np.abs(ref) + 1e-6).all()
    B.gdn_attn_prefill_weights(q, k, lse, w, table_d, cu_d)
    got = w.cpu().numpy()
    wn = C.prefill_weights(np64(q), np64(k), rl, np.full(got.shape, np.nan), table.numpy(), cu)
    fin = ~np.isnan(wn)
    assert np.allclose(got[fin], wn[fin], rtol=1e-3, atol=1e-6) and np.isnan(got[~fin]).all()

    raw = lambda x: as_bytes(x) if bits == 8 else x.view(torch.int16).cpu().numpy()
    before = [raw(caches["k_cache"]), raw(caches["v_cache"]), got]
    before += [scales[s].cpu().numpy() for s in ("k_scale", "v_scale")] if bits == 8 else [None, None]
    new_lens, kept = B.gdn_attn_evict(caches["k_cache"], caches["v_cache"], w, table_d, kv, new.cuda(), keep, recent, **scales)
    dst, wl, wk = C.evict(before[0], before[1], before[2], table.numpy(), lens, new.numpy(), keep, recent, before[3], before[4])
    assert np.array_equal(kept.cpu().numpy(), wk) and new_lens.tolist() == wl.tolist() == [48, 40]
    assert np.array_equal(raw(caches["k_cache"]), dst[0]) and np.array_equal(raw(caches["v_cache"]), dst[1])

    tables, at = new.cuda(), [130, 40]  # positions go on where the prompts ended
    for step in range(12):
        new_lens = new_lens + 1
        p = torch.tensor(at, dtype=torch.int32).repeat(3, 1)
        at = [a + 1 for a in at]
        q, k, v = front(randn(g, N, (H + 2 * Hk) * D, mul=2.0), p, new_lens, i32([0, 1, 2]), tables)
        w0 = w.cpu().numpy()
        out = B.gdn_attn_decode(q, caches["k_cache"], caches["v_cache"], tables, new_lens, weights=w, **scales)
        if bits == 8:
            kvals, vvals = (C.held(as_bytes(caches[c]), scales[s].cpu().numpy())
                            for c, s in (("k_cache", "k_scale"), ("v_cache", "v_scale")))
        else:
            kvals, vvals = np64(caches["k_cache"]), np64(caches["v_cache"])
        ref, mag, _ = A.decode(np64(q)[:, None], kvals, vvals, new.numpy(), new_lens.tolist())
        o = np64(out)[:, None]
        assert (np.abs(o - ref) <= REL * mag + 2.0 ** -8 * np.abs(ref) + 1e-6).all()
        want = C.decode_weights(np64(q)[:, None], kvals, new.numpy(), new_lens.tolist(), w0)
        g1 = w.cpu().numpy()
        fin = ~np.isnan(want)
        assert np.allclose(g1[fin], want[fin], rtol=1e-4, atol=1e-6)


# ---------------------------------------------------------------- what single calls got wrong
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 5, 7, 10, 15, 20])  # each number of row tiles and warps for 3 tokens
@pytest.mark.parametrize("length", [18, 34])  # the block behind is a half of 32 keys, or 32 of its own
def test_decode8_scales_of_later_tokens_have_no_influence(length, G, D):
    """Row i does not see the tokens behind it, nor the scales of a block that holds only such
    tokens: with a scale there that is no number, or infinite, row 0's output stays as it is."""
    g = torch.Generator().manual_seed(length + G)
    H, nq = 2 * G, 3
    kb, ks = random_cache8(g, 3, 2, 16, D)
    vb, vs = random_cache8(g, 3, 2, 16, D)
    q = randn(g, 1, nq, H, D)
    table, last = i32([[2, 0, 1]]), [2, 0, 1][length // 16]

    def run(weights=None):
        return B.gdn_attn_decode(q.cuda(), kb.cuda().view(F8), vb.cuda().view(F8), table, i32([length]),
                                 k_scale=ks.cuda(), v_scale=vs.cuda(), out_dtype=F32, return_lse=True,
                                 weights=weights)
    keep = ks[last].clone()
    want, want_lse = run()
    assert want.isfinite().all()
    w = torch.zeros(3, 2, 16, device="cuda")
    run(w)
    for bad in (float("nan"), float("inf")):
        vs[last] = bad
        got, lse = run()
        assert torch.equal(got[:, 0], want[:, 0]) and torch.equal(lse, want_lse)
        assert not got[:, 1:].isfinite().any()  # (rows that see it)
        w2 = torch.zeros_like(w)
        assert torch.equal(run(w2)[0][:, 0], want[:, 0]) and torch.equal(w2, w)
        ks[last] = bad
        got, lse = run()
        assert torch.equal(got[:, 0], want[:, 0]) and torch.equal(lse[:, 0], want_lse[:, 0])
        ks[last] = keep


def evict_called_with(monkeypatch, columns=0, skew=0):
    """The calls that follow get page tables of at least `columns` columns, and weights that begin
    `skew` floats past a 16-byte boundary."""
    real = B.gdn_attn_evict

    def call(k, v, w, table, *rest, **kw):
        wide = torch.full((table.shape[0], max(columns, table.shape[1])), -1, dtype=torch.int32, device="cuda")
        wide[:, :table.shape[1]] = table
        room = torch.empty(w.numel() + 4, device="cuda")
        there = room[skew:skew + w.numel()].view(w.shape)
        assert room.data_ptr() % 16 == 0
        there.copy_(w)
        out = real(k, v, there, wide, *rest, **kw)
        w.copy_(there)
        return out
    monkeypatch.setattr(B, "gdn_attn_evict", call)


def test_evict_rows_of_any_length_in_a_wide_table(monkeypatch):
    """What a row takes goes by its own length: either side of each change, in one call."""
    evict_called_with(monkeypatch, columns=200)  # of 256 tokens
    for recent in (0, 17):
        run_evict([300, 0, 8192 + recent, 8193 + recent, 32768 + recent, 32769 + recent, 250, 251], 1, 64, 256, 250,
                  recent, seed=recent)
    run_evict([40000, 9, 33000], 2, 64, 256, 9000, 100, 8, change=lambda w: (w * 3).round())
    run_evict([8000, 32000], 1, 64, 256, 7990, 0, change=torch.ones_like)
    evict_called_with(monkeypatch, columns=2049)  # of 16 tokens
    run_evict([700, 100, 513, 9000], 2, 64, 16, 90, 7)


@pytest.mark.parametrize("skew", [1, 2, 3])
def test_evict_weights_that_begin_anywhere(monkeypatch, skew):
    """Weights are 4-byte aligned; from a 16-byte boundary on they are read four at a time, else singly."""
    evict_called_with(monkeypatch, skew=skew)
    for longest in (2048, 4096, 8192, 16384, 32768):
        run_evict([longest, 9, longest - 1, longest // 2 + 3], 1, 64, 256, longest // 3, 17, seed=longest)
    run_evict([700, 100, 513], 2, 64, 16, 90, 7, 8)
    evict_called_with(monkeypatch, columns=200, skew=skew)
    run_evict([8000, 9000, 17000, 33000, 40], 1, 64, 256, 50, 7)


@pytest.mark.parametrize("bits", [8, 16])
def test_weights_that_begin_anywhere(monkeypatch, bits):
    """As above, of a decode step and of a prompt."""
    decode, prompt = B.gdn_attn_decode, B.gdn_attn_prefill_weights

    def skewed(w):
        room = torch.empty(w.numel() + 4, device="cuda")
        there = room[1:1 + w.numel()].view(w.shape)
        there.copy_(w)
        return there

    def step(*a, weights=None, **kw):
        there = skewed(weights)
        out = decode(*a, weights=there, **kw)
        weights.copy_(there)
        return out

    def whole(q, k, lse, weights, *a, **kw):
        there = skewed(weights)
        prompt(q, k, lse, there, *a, **kw)
        weights.copy_(there)
    monkeypatch.setattr(B, "gdn_attn_decode", step)
    monkeypatch.setattr(B, "gdn_attn_prefill_weights", whole)
    run_decode([70, 1, 150], 6, 2, 64, 16, bits=bits, weights=True)
    run_decode([5, 33, 100], 4, 2, 128, 32, nq=4, bits=bits, weights=True)
    run_prompt([300, 20], 4, 2, 128)


@pytest.mark.parametrize("longest", [600, 3000, 8000, 16000, 32000, 40000])
def test_evict_pages_that_do_not_exist_are_reported_where_nothing_of_them_stays(longest):
    page, keep, recent = 256, 20, 4
    cols = -(-longest // page)
    for bad in (-1, cols + 1):
        table = torch.arange(cols, dtype=torch.int32)[None].cuda()
        k = torch.ones(cols + 1, 1, page, 64, dtype=BF, device="cuda")
        w = torch.rand(cols + 1, 1, page, device="cuda") + 1
        w[cols - 2] += 2  # the tokens that stay are of this page, the last ones of the last
        status = new_status()
        run = lambda: B.gdn_attn_evict(k, k, w, table, i32([longest]), i32([[cols]]), keep, recent, status=status)
        want = run()[1]
        assert status.item() == 0
        table[0, 0] = bad
        got = run()[1]
        assert status.item() == 64 and torch.equal(got, want)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("nq, G", [(1, 4), (3, 2), (4, 8), (8, 8)])  # one, two and four row tiles
def test_decode_with_weights_keeps_sixteen_bits_of_them(nq, G, D):
    """Over a bf16 cache, 32-bit outputs. Each weight goes into the product in two bf16 parts, off by
    2^-16 of it at most; scores and exp add weight_slack's part (that amount for the weight, as much for
    its denominator), sums in 32 bits of at most 64 products a part and their merge 2^-18. The weights
    rounded to bf16 alone (2^-9 each) would pass it."""
    g = torch.Generator().manual_seed(nq + D)
    H, page, lens = 2 * G, 16, [nq + 2, 9, 33, 64]
    N = len(lens)
    q = randn(g, N, nq, H, D, mul=0.2)
    table, n_pages, _ = pages_for(g, [-(-n // page) for n in lens], 1)
    k, v = randn(g, n_pages, 2, page, D), randn(g, n_pages, 2, page, D)
    w = torch.zeros(n_pages, 2, page, device="cuda")
    out = B.gdn_attn_decode(q.cuda(), k.cuda(), v.cuda(), table.cuda(), i32(lens), out_dtype=F32, weights=w)
    ref, mag, _ = A.decode(np64(q), np64(k), np64(v), table.numpy(), lens)
    tol = 2.0 ** -16 + 2.0 ** -18 + 2 * weight_slack(q, np64(k), D, D ** -0.5)
    assert tol < 2.0 ** -11
    assert (np.abs(np64(out) - ref) <= tol * mag + 1e-9).all()


@pytest.mark.parametrize("nq", [1, 3])
def test_decode_with_weights_over_infinite_values(nq):
    """An infinite value is infinite for the rows that see it, whatever the bits of its weight (equal
    scores here: weights of 1, which leave no rest), and nothing for the others."""
    g = torch.Generator().manual_seed(3)
    k, v = torch.zeros(2, 1, 16, 64, dtype=BF), randn(g, 2, 1, 16, 64)
    table, w = i32([[1, 0]]), torch.zeros(2, 1, 16, device="cuda")
    q = randn(g, 1, nq, 2, 64)
    for scores in (0.0, 1.0):
        k[:] = scores * randn(g, 2, 1, 16, 64)
        x = v.clone()
        x[1, 0, 3, 5], x[1, 0, 9, 6], x[0, 0, 3, 7] = float("inf"), float("-inf"), float("inf")
        out = B.gdn_attn_decode(q.cuda(), k.cuda(), x.cuda(), table, i32([20]), out_dtype=F32, weights=w)
        assert (out[..., 5] == float("inf")).all() and (out[..., 6] == float("-inf")).all()
        assert (out[0, -1, :, 7] == float("inf")).all() and out[0, :-1, :, 7].isfinite().all()
        rest = [c for c in range(64) if c not in (5, 6, 7)]
        assert out[..., rest].isfinite().all()
