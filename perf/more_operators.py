"""The cache of a long conversation as workloads: the front end with rotary positions of several
axes, a paged cache in 8 bits (append, decode attention), the attention weight that keys gather
(while decoding, and from a prompt's rows), and eviction by that weight.

`run` computes an operator in its plain form (elementary torch operations in 32 bits, one
rounding at the end) or, where `own` is true, through the package's entry points. `exact`
evaluates the definitions in 64 bits. Caches in 8 bits are returned as they are held, as float8
values, with their scales beside them.
"""
import math
import random

import torch

own = False

PAGE_SIZES = (16, 32, 64, 128, 256)
BLOCK = 16  # tokens of the 8-bit cache that share a scale


# ---------------------------------------------------------------- cases
def listed():
    return [
        # A decode step of a full batch whose sequences hold images or were cut: their positions
        # are not their places in the cache. Nothing but latency.
        dict(name="front_axes_step_64", op="front", N=64, lo=1, hi=1, past=8190, H=32, Hk=8, D=128,
             rot=128, n_axes=3, axes="sections", interleaved=False, page=64, dense=False, lens_seed=1),
        # A prompt of text and images, a quarter of the head rotated, the axes dealt out in turn;
        # k and v kept dense for the prompt's own attention.
        dict(name="front_axes_prompt_4096", op="front", N=1, lo=4096, hi=4096, past=0, H=16, Hk=2, D=128,
             rot=32, n_axes=3, axes="cyclic", interleaved=True, page=64, dense=True, lens_seed=2),
        # The same full batch's new keys and values, one token each, into the 8-bit cache: most
        # blocks hold earlier tokens.
        dict(name="append8_step_64", op="append8", N=64, lo=1, hi=1, past=8190, Hk=8, D=128, page=64,
             lens_seed=3),
        # Packed prompts of uneven lengths that go on from what the cache holds.
        dict(name="append8_ragged_8", op="append8", N=8, lo=1, hi=2048, past=777, Hk=8, D=128, page=64,
             lens_seed=4),
        # One conversation's next token over its own context in 8 bits: latency, one long axis.
        dict(name="decode8_1", op="decode8", N=1, nq=1, lo=8191, hi=8191, H=16, Hk=4, D=128, page=16,
             lens_seed=5),
        # A batch's next tokens, contexts of very different lengths, in 8 bits.
        dict(name="decode8_64", op="decode8", N=64, nq=1, lo=1, hi=8192, H=32, Hk=8, D=128, page=64,
             lens_seed=6),
        # A batch's next tokens over the bf16 cache, with the weight that each key gets.
        dict(name="decode_weights_64", op="weights", bits=16, N=64, nq=1, lo=1, hi=4096, H=32, Hk=8, D=128,
             page=64, lens_seed=7),
        # A few tokens of each sequence to verify, head size 64, an odd group, 8 bits, with weights.
        dict(name="decode8_weights_verify_8", op="weights", bits=8, N=8, nq=4, lo=1000, hi=8000, H=20, Hk=4,
             D=64, page=32, lens_seed=8),
        # The weight that a whole prompt's rows give its keys, at the length of the delta-rule
        # workloads.
        dict(name="prompt_weights_4096", op="prompt", N=1, lo=4096, hi=4096, H=16, Hk=4, D=128, page=64,
             window=0, lens_seed=9),
        # Packed prompts of uneven lengths.
        dict(name="prompt_weights_ragged_8", op="prompt", N=8, lo=1, hi=2048, H=32, Hk=8, D=128, page=16,
             window=0, lens_seed=10),
        # A batch cut to a budget, the last tokens kept; some sequences are shorter than it.
        dict(name="evict_64", op="evict", bits=16, N=64, lo=1, hi=4096, Hk=8, D=128, page=64, keep=1024,
             recent=128, lens_seed=11),
        # One long conversation in 8 bits cut to a quarter, an odd budget.
        dict(name="evict8_1", op="evict", bits=8, N=1, lo=16383, hi=16383, Hk=4, D=128, page=16, keep=4001,
             recent=33, lens_seed=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("front", "append8", "decode8", "weights", "prompt", "evict"))
    while True:
        Hk = rng.choice((1, 2, 3, 4, 8))
        G = rng.choice((1, 2, 3, 4, 5, 6, 7, 8, 16))
        D = rng.choice((64, 128, 128))
        c = dict(op=op, Hk=Hk, D=D, page=rng.choice(PAGE_SIZES), lens_seed=rng.randrange(1 << 20))
        if op in ("front", "append8"):
            step = rng.random() < 0.4
            N = _log(rng, 1, 256) if step else _log(rng, 1, 32)
            hi = 1 if step else _log(rng, 2, 8192)
            c.update(N=N, lo=1, hi=hi, past=rng.choice((0, _log(rng, 1, 8192))))
            if op == "front":
                c.update(H=Hk * G, rot=rng.choice((16, 32, D // 2, D)), n_axes=rng.choice((1, 2, 3, 3, 4)),
                         axes=rng.choice(("sections", "cyclic")), interleaved=rng.random() < 0.5,
                         dense=not step)
            if N * hi <= 32768 and N * (c["past"] + hi) * Hk * D <= 1 << 28:
                return c
        elif op in ("decode8", "weights"):
            N, hi = _log(rng, 1, 128), _log(rng, 1, 16384)
            nq = rng.choice((1, 1, 1, 2, 3, 5, 8))
            c.update(N=N, nq=nq, H=Hk * G, lo=max(nq, hi // rng.choice((1, 2, 1000000))), hi=max(nq, hi))
            if op == "weights":
                c["bits"] = rng.choice((16, 8))
            if nq * G <= 64 and N * c["hi"] * Hk <= 1 << 21 and N * nq * c["H"] * c["hi"] <= 1 << 27:
                return c
        elif op == "prompt":
            N, hi = _log(rng, 1, 32), _log(rng, 1, 8192)
            c.update(N=N, H=Hk * G, lo=max(1, hi // rng.choice((1, 2, 8, 1000000))), hi=hi,
                     window=rng.choice((0, 0, 0, _log(rng, 1, 512))))
            if N * hi * hi * c["H"] <= 8192 * 8192 * 8 and N * hi <= 65536:
                return c
        else:
            N, hi = _log(rng, 1, 64), _log(rng, 16, 32768)
            keep = max(2, _log(rng, 1, hi))
            c.update(N=N, lo=max(1, hi // rng.choice((1, 2, 1000000))), hi=hi, keep=keep,
                     recent=rng.choice((0, keep // 8, rng.randint(0, keep))), bits=rng.choice((16, 8)))
            if N * hi * Hk <= 1 << 21:
                return c


def _lens(case):
    r = random.Random(case["lens_seed"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["N"])]


def _pasts(case):
    r = random.Random(case["lens_seed"] + 1)
    return [r.randint((case["past"] + 1) // 2, case["past"]) for _ in range(case["N"])]


def work(case):
    op, Hk, D, lens = case["op"], case["Hk"], case["D"], _lens(case)
    T = sum(lens)
    if op == "front":
        H = case["H"]
        table = 4 * case["rot"] * T + 4 * case["n_axes"] * T  # a row's pairs and the positions
        return {"bytes": 2 * T * (2 * H + 2 * Hk) * D + 4 * T * Hk * D * (2 if case["dense"] else 1) + table,
                "flops": 8 * T * (H + Hk) * D}
    if op == "append8":
        scales = 8 * Hk * sum(-(-n // BLOCK) for n in lens)
        return {"bytes": 2 * T * Hk * D * 3 + scales, "flops": 4 * T * Hk * D}
    if op in ("decode8", "weights"):
        N, nq, H = case["N"], case["nq"], case["H"]
        key = 4 * D if case.get("bits", 8) == 16 else 2 * D + 8 / BLOCK
        if op == "weights":
            key += 8
        pairs = sum(nq * n - nq * (nq - 1) // 2 for n in lens)
        return {"bytes": Hk * T * key + 4 * N * nq * H * D, "flops": 4 * D * H * pairs}
    if op == "prompt":
        H, w = case["H"], case["window"]
        rows = [(n, min(n, w) if w else n) for n in lens]
        pairs = sum(r * n - r * (r - 1) // 2 for n, r in rows)
        return {"bytes": 2 * sum(r for _, r in rows) * H * (D + 2) + 2 * T * Hk * D + 4 * T * Hk,
                "flops": 2 * D * H * pairs}
    kept = sum(min(n, case["keep"]) for n in lens)
    move = (4 * D if case["bits"] == 16 else 2 * D + 8 / BLOCK) + 4
    return {"bytes": Hk * (4 * T + 2 * kept * move + 4 * kept), "flops": 2 * Hk * T}


# ---------------------------------------------------------------- inputs
def _pages(g, counts, spare=0):
    """A page table [N, width] of physical pages in scattered order; a row's last page stands for
    what is past it. Also the number of pages, and `spare` pages more that no sequence has."""
    n_pages = sum(counts) + spare
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    count = torch.tensor(counts, device="cuda")
    first = torch.cumsum(count, 0) - count
    i = torch.arange(max(counts), device="cuda")[None, :]
    table = perm[first[:, None] + torch.minimum(i, (count - 1)[:, None])].contiguous()
    return table, n_pages, perm[sum(counts):]


def _scale_of(top):
    """The least power of two s with top <= 448 s (from 2^-100 on)."""
    m, e = torch.frexp(top)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-100)
    return torch.where(top > 0, torch.exp2(e.double()), 2.0 ** -100).float()


def _held8(x):
    """[pages, Hk, page, D] in 32 bits -> float8 values and scales [pages, Hk, page / BLOCK]."""
    p, h, n, d = x.shape
    s = _scale_of(x.view(p, h, n // BLOCK, BLOCK * d).abs().amax(-1))
    return (x.view(p, h, n // BLOCK, BLOCK, d) / s[..., None, None]).to(torch.float8_e4m3fn).view(x.shape), s


def _positions(case, seed, kv):
    """[n_axes, T]: text (all axes alike) with images between (rows and columns of a grid on the
    last two axes); a position is behind the token's place where images stood before it."""
    r = random.Random(int(seed) * 7919 + case["lens_seed"])
    A, parts = case["n_axes"], []
    for n, length in zip(_lens(case), kv):
        at = r.randint(0, length - n)
        while n > 0:
            k = min(n, r.randint(1, 700))
            i = torch.arange(k)
            if r.random() < 0.5 and A > 1:
                width = r.randint(4, 32)
                p = torch.full((A, k), at)
                p[-1] += i % width
                p[-2] += i // width
                at += max(width, k // width + 1)
            else:
                p = (at + i).expand(A, k)
                at += k
            parts.append(p)
            n -= k
    return torch.cat(parts, 1).to(torch.int32).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, Hk, D, N, page, lens = case["op"], case["Hk"], case["D"], case["N"], case["page"], _lens(case)
    T = sum(lens)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    def i32(x):
        return torch.tensor(x, device="cuda", dtype=torch.int32)

    def caches(n_pages, bits):
        if bits == 16:
            return dict(k_cache=normal(n_pages, Hk, page, D), v_cache=normal(n_pages, Hk, page, D))
        c = {}
        for x in ("k", "v"):
            # heads, and tokens among them, of different sizes
            size = torch.exp2(normal(n_pages, Hk, page, 1, dtype=torch.float32))
            c[x + "_cache"], c[x + "_scale"] = _held8(normal(n_pages, Hk, page, D, dtype=torch.float32) * size)
        return c

    cu = i32([0] + lens).cumsum(0).to(torch.int32)
    if op in ("front", "append8"):
        kv = [p + n for p, n in zip(_pasts(case), lens)]
        table, n_pages, _ = _pages(g, [-(-n // page) for n in kv])
        s = dict(case=case, cu=cu, kv_lens=i32(kv), table=table)
        if op == "append8":
            s.update(caches(n_pages, 8), k=normal(T, Hk, D), v=normal(T, Hk, D) * 3.0)
            return s
        H, rot, A = case["H"], case["rot"], case["n_axes"]
        i = torch.arange(rot // 2, device="cuda")
        axes = i % A if case["axes"] == "cyclic" else i * A // (rot // 2)
        freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        angle = torch.arange(max(kv) + 1024, device="cuda", dtype=torch.float64)[:, None] * freq
        s.update(caches(n_pages, 16), x=normal(T, (H + 2 * Hk) * D) * 2.0, axes=axes.to(torch.uint8),
                 positions=_positions(case, seed, kv), q_weight=1.0 + 0.1 * normal(D, dtype=torch.float32),
                 k_weight=1.0 + 0.1 * normal(D, dtype=torch.float32),
                 rope=torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32), eps=1e-6)
        return s
    if op == "evict":
        keep = case["keep"]
        fresh = [-(-min(n, keep) // page) for n in lens]
        table, n_pages, spare = _pages(g, [-(-n // page) for n in lens], sum(fresh))
        first = torch.tensor(fresh, device="cuda").cumsum(0) - torch.tensor(fresh, device="cuda")
        i = torch.arange(-(-keep // page), device="cuda")[None, :]
        new = spare[first[:, None] + torch.minimum(i, torch.tensor(fresh, device="cuda")[:, None] - 1)]
        # weights over many powers of ten, a tenth of them equal (never seen since)
        w = torch.exp(3.0 * normal(n_pages, Hk, page, dtype=torch.float32))
        w[torch.rand(w.shape, generator=g, device="cuda") < 0.1] = 0.0
        return dict(case=case, table=table, new_table=new.contiguous(), kv_lens=i32(lens), weights=w,
                    **caches(n_pages, case["bits"]))
    H = case["H"]
    if op == "prompt":
        table, n_pages, _ = _pages(g, [-(-n // page) for n in lens])
        q, k = normal(T, H, D), normal(T, Hk, D)
        lse = torch.empty(T, H, device="cuda")
        b = 0
        for n in lens:  # what the prompt's attention has returned
            i = torch.arange(n, device="cuda")
            for h in range(H):
                x = q[b:b + n, h].float() @ k[b:b + n, h * Hk // H].float().T * D ** -0.5
                lse[b:b + n, h] = x.masked_fill_(i[None, :] > i[:, None], float("-inf")).logsumexp(-1)
            b += n
        return dict(case=case, q=q, k=k, lse=lse, cu=cu, table=table, longest=max(lens),
                    weights=torch.rand(n_pages, Hk, page, generator=g, device="cuda"))
    nq = case["nq"]
    table, n_pages, _ = _pages(g, [-(-n // page) for n in lens])
    s = dict(case=case, q=normal(*((N, H, D) if nq == 1 else (N, nq, H, D))), table=table, kv_lens=i32(lens),
             **caches(n_pages, case.get("bits", 8)))
    if op == "weights":  # gathered by the steps before
        s["weights"] = torch.rand(n_pages, Hk, page, generator=g, device="cuda") * 4.0
    return s


# ---------------------------------------------------------------- the operators
def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _own_front(s):
    from gated_delta_rule_chunk_gb300 import binding as B
    c = s["case"]
    q, k, v = B.gdn_attn_front(s["x"], c["H"], c["Hk"], c["D"], q_weight=s["q_weight"],
                               k_weight=s["k_weight"], norm_eps=s["eps"], rope=s["rope"],
                               interleaved=c["interleaved"], cu_seqlens=s["cu"], kv_lens=s["kv_lens"],
                               page_table=s["table"], k_cache=s["k_cache"], v_cache=s["v_cache"],
                               output_kv=c["dense"], positions=s["positions"], rope_axes=s["axes"])
    return dict(q=q, k=k, v=v, k_cache=s["k_cache"], v_cache=s["v_cache"])


def _own_append8(s):
    from gated_delta_rule_chunk_gb300 import binding as B
    B.gdn_attn_append8(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                       kv_lens=s["kv_lens"], cu_seqlens=s["cu"])
    return {x: s[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _own_decode(s):
    from gated_delta_rule_chunk_gb300 import binding as B
    out = B.gdn_attn_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"],
                            k_scale=s.get("k_scale"), v_scale=s.get("v_scale"), weights=s.get("weights"))
    return dict(out=out, weights=s.get("weights"))


def _own_prompt(s):
    from gated_delta_rule_chunk_gb300 import binding as B
    B.gdn_attn_prefill_weights(s["q"], s["k"], s["lse"], s["weights"], s["table"], cu_seqlens=s["cu"],
                               window=s["case"]["window"])
    return s["weights"]


def _own_evict(s):
    from gated_delta_rule_chunk_gb300 import binding as B
    c = s["case"]
    lens, kept = B.gdn_attn_evict(s["k_cache"], s["v_cache"], s["weights"], s["table"], s["kv_lens"],
                                  s["new_table"], c["keep"], recent=c["recent"], k_scale=s.get("k_scale"),
                                  v_scale=s.get("v_scale"))
    return dict(lens=lens, kept=kept, **{x: s.get(x) for x in ("k_cache", "v_cache", "k_scale", "v_scale",
                                                               "weights")})


def _norm_rotate(x, weight, eps, cos, sin, interleaved):
    """x [T, heads, D] fp32; cos, sin [T, rot / 2]."""
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight
    h = cos.shape[1]
    cos, sin = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :h], x[..., h:2 * h]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., 2 * h:]], -1)


def _places(s):
    """Sequence and place in the cache of each of the call's tokens."""
    t = torch.arange(int(s["x" if "x" in s else "k"].shape[0]), device=s["cu"].device)
    n = torch.searchsorted(s["cu"][1:], t, right=True)
    return n, (s["kv_lens"] - s["cu"][1:])[n] + t


def _plain_front(s):
    c = s["case"]
    H, Hk, D, page, half = c["H"], c["Hk"], c["D"], c["page"], c["rot"] // 2
    x = s["x"].float()
    T, dt = x.shape[0], s["k_cache"].dtype
    n, at = _places(s)
    i = torch.arange(half, device=x.device)
    row = s["positions"].long().T[:, s["axes"].long()]  # [T, rot / 2]
    cos, sin = s["rope"][row, i], s["rope"][row, half + i]
    q, k, v = (y.view(T, -1, D) for y in x.split([H * D, Hk * D, Hk * D], 1))
    q = _norm_rotate(q, s["q_weight"], s["eps"], cos, sin, c["interleaved"]).to(dt)
    k = _norm_rotate(k, s["k_weight"], s["eps"], cos, sin, c["interleaved"]).to(dt)
    v = v.to(dt)
    pg = s["table"][n, at // page].long()
    s["k_cache"][pg, :, at % page] = k
    s["v_cache"][pg, :, at % page] = v
    return dict(q=q, k=k if c["dense"] else None, v=v if c["dense"] else None, k_cache=s["k_cache"],
                v_cache=s["v_cache"])


def _plain_append8(s):
    c = s["case"]
    Hk, D, page = c["Hk"], c["D"], c["page"]
    n, at = _places(s)
    before = s["kv_lens"] - (s["cu"][1:] - s["cu"][:-1])  # tokens that the cache holds already
    pg = s["table"][n, at // page].long()
    block = pg * (page // BLOCK) + at % page // BLOCK  # one number for each block of the cache
    had = at // BLOCK * BLOCK < before[n]  # the token's block holds earlier ones
    # each sequence's block that holds its last earlier token, and its rows
    start = (before // BLOCK * BLOCK).long()
    row = start[:, None] + torch.arange(BLOCK, device=at.device)  # [N, BLOCK]
    seq = torch.arange(c["N"], device=at.device)
    page0 = s["table"][seq, start // page].long()
    old_row = (row < before[:, None])[:, :, None, None]
    out = {}
    for x in ("k", "v"):
        new, cache, scale = s[x].float(), s[x + "_cache"], s[x + "_scale"]
        old = scale[pg, :, at % page // BLOCK]
        top = torch.zeros(scale.shape[0] * scale.shape[2], Hk, device=new.device)
        top.scatter_reduce_(0, block[:, None].expand(-1, Hk), new.abs().amax(-1), "amax")
        grown = torch.maximum(_scale_of(top[block]), torch.where(had[:, None], old, 0.0))
        old0 = scale[page0, :, start % page // BLOCK]  # [N, Hk]
        scale[pg, :, at % page // BLOCK] = grown
        ratio = old0 / scale[page0, :, start % page // BLOCK]
        bits = cache.view(torch.uint8)
        held = bits[page0[:, None], :, row % page]  # [N, BLOCK, Hk, D]
        again = (held.view(cache.dtype).float() * ratio[:, None, :, None]).to(cache.dtype).view(torch.uint8)
        bits[page0[:, None], :, row % page] = torch.where(old_row, again, held)
        bits[pg, :, at % page] = (new / grown[..., None]).to(cache.dtype).view(torch.uint8)
        out[x + "_cache"], out[x + "_scale"] = cache, scale
    return out


def _keys(s, x):
    """The sequences' keys or values in 32 bits: [N, Hk, width * page, D]."""
    table = s["table"].long()
    if s[x + "_cache"].dtype == torch.bfloat16:
        rows = s[x + "_cache"][table].float()  # [N, width, Hk, page, D]
    else:
        rows = s[x + "_cache"].view(torch.uint8)[table].view(s[x + "_cache"].dtype).float()
        rows *= s[x + "_scale"][table].repeat_interleave(BLOCK, -1)[..., None]
    return rows.transpose(1, 2).reshape(table.shape[0], rows.shape[2], -1, rows.shape[-1])


def _plain_decode(s):
    c, q = s["case"], s["q"]
    N, nq, H, Hk, D, page = c["N"], c["nq"], c["H"], c["Hk"], c["D"], c["page"]
    G = H // Hk
    rows = (q.float() * D ** -0.5).view(N, nq, Hk, G, D).transpose(1, 2).reshape(N, Hk, nq * G, D)
    w = rows @ _keys(s, "k").transpose(-1, -2)
    w = w.view(N, Hk, nq, G, -1)
    j = torch.arange(w.shape[-1], device=q.device)
    lens = s["kv_lens"].long()
    last = lens[:, None] - nq + torch.arange(nq, device=q.device)
    w.masked_fill_(~(j <= last[:, None, :, None, None]), float("-inf"))
    w.sub_(w.amax(-1, keepdim=True)).exp_()  # every row sees a key
    w.div_(w.sum(-1, keepdim=True))
    out = w.view(N, Hk, nq * G, -1) @ _keys(s, "v")
    out = out.view(N, Hk, nq, G, D).transpose(1, 2).reshape(q.shape).to(q.dtype)
    if "weights" not in s:
        return dict(out=out, weights=None)
    gained = w.sum((2, 3)).permute(0, 2, 1)  # [N, keys, Hk]
    n, j = (j[None, :] < lens[:, None]).nonzero(as_tuple=True)
    pg = s["table"][n, j // page].long()
    known = torch.where((j < lens[n] - nq)[:, None], s["weights"][pg, :, j % page], 0.0)
    s["weights"][pg, :, j % page] = known + gained[n, j]
    return dict(out=out, weights=s["weights"])


def _plain_prompt(s):
    c, q, k, cu, L = s["case"], s["q"], s["k"], s["cu"].long(), s["longest"]
    T, H, D = q.shape
    Hk, N, page = k.shape[1], cu.numel() - 1, c["page"]
    t = torch.arange(T, device=q.device)
    n = torch.searchsorted(cu[1:], t, right=True)
    i = t - cu[n]

    def padded(x, fill=0.0):  # [T, heads, ...] -> [N, heads, L, ...] in 32 bits
        y = x.new_full((N, L) + x.shape[1:], fill, dtype=torch.float32)
        y[n, i] = x.float()
        return y.transpose(1, 2)

    lse = s["lse"]
    if c["window"]:  # rows before the window give nothing
        lse = torch.where((i >= (cu[1:] - cu[:-1])[n] - c["window"])[:, None], lse, float("inf"))
    rows = (padded(q) * D ** -0.5).reshape(N, Hk, H // Hk * L, D)
    w = (rows @ padded(k).transpose(-1, -2)).view(N, Hk, H // Hk, L, L)
    w.sub_(padded(lse, float("inf")).reshape(N, Hk, H // Hk, L, 1)).exp_()
    a = torch.arange(L, device=q.device)
    w.masked_fill_(a[None, :] > a[:, None], 0.0)
    total = w.sum((2, 3))  # [N, Hk, L]
    s["weights"][s["table"][n, i // page].long(), :, i % page] = total[n, :, i]
    return s["weights"]


def _plain_evict(s):
    c = s["case"]
    page, keep, recent = c["page"], c["keep"], c["recent"]
    table, new, w = s["table"].long(), s["new_table"].long(), s["weights"]
    N, Hk = table.shape[0], w.shape[1]
    lens = s["kv_lens"].long()[:, None, None]
    rank = w[table].transpose(1, 2).reshape(N, Hk, -1)
    j = torch.arange(rank.shape[-1], device=w.device)
    rank = torch.where(j >= lens - recent, float("inf"), rank)
    rank = torch.where(j >= lens, float("-inf"), rank)
    kept = rank.argsort(dim=-1, descending=True, stable=True)[..., :keep].sort(-1).values
    kept = torch.nn.functional.pad(kept, (0, keep - kept.shape[-1]), value=1 << 30)
    there = kept < lens  # the others come last
    # places that no token takes repeat the first one's copy
    src = torch.where(there, kept, kept[..., :1])
    dst = torch.where(there, torch.arange(keep, device=w.device), 0)
    n, h = torch.arange(N, device=w.device)[:, None, None], torch.arange(Hk, device=w.device)[:, None]
    at, to = (table[n, src // page], h, src % page), (new[n, dst // page], h, dst % page)
    if "k_scale" in s:
        for x in ("k", "v"):
            cache, scale = s[x + "_cache"], s[x + "_scale"]
            old = scale[at[0], h, at[2] // BLOCK]
            over = torch.nn.functional.pad(torch.where(there, old, 0.0), (0, -keep % BLOCK))
            most = over.view(N, Hk, -1, BLOCK).amax(-1).repeat_interleave(BLOCK, -1)[..., :keep]
            most = torch.where(there, most, most[..., :1])
            bits = cache.view(torch.uint8)
            rows = bits[at].view(cache.dtype).float() * (old / most)[..., None]
            bits[to] = rows.to(cache.dtype).view(torch.uint8)
            scale[to[0], h, to[2] // BLOCK] = most
    else:
        for x in ("k_cache", "v_cache"):
            s[x][to] = s[x][at]
    w[to] = w[at]
    return dict(lens=lens.flatten().clamp(max=keep).to(torch.int32),
                kept=torch.where(there, kept, -1).to(torch.int32),
                **{x: s.get(x) for x in ("k_cache", "v_cache", "k_scale", "v_scale", "weights")})


_own = dict(front=_own_front, append8=_own_append8, decode8=_own_decode, weights=_own_decode,
            prompt=_own_prompt, evict=_own_evict)
_plain = dict(front=_plain_front, append8=_plain_append8, decode8=_plain_decode, weights=_plain_decode,
              prompt=_plain_prompt, evict=_plain_evict)


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return dict(front=_exact_front, append8=_exact_append8, decode8=_exact_decode, weights=_exact_decode,
                prompt=_exact_prompt, evict=_exact_evict)[case["op"]](s)


def _exact_front(s):
    c = s["case"]
    H, Hk, D, page, rot = c["H"], c["Hk"], c["D"], c["page"], c["rot"]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    qs, ks, vs = [], [], []
    cu, kv = s["cu"].tolist(), s["kv_lens"].tolist()
    first = torch.arange(0, rot, 2) if c["interleaved"] else torch.arange(rot // 2)
    second = first + (1 if c["interleaved"] else rot // 2)
    axes = s["axes"].tolist()
    for n in range(c["N"]):
        x = s["x"][cu[n]:cu[n + 1]].double().view(-1, H + 2 * Hk, D)
        p = torch.arange(kv[n] - x.shape[0], kv[n], device=x.device)
        where = s["positions"][:, cu[n]:cu[n + 1]].long()
        turn = torch.stack([torch.complex(s["rope"][where[a], i].double(), s["rope"][where[a], rot // 2 + i].double())
                            for i, a in enumerate(axes)], -1)[:, None, :]
        parts = []
        for y, w in ((x[:, :H], s["q_weight"]), (x[:, H:H + Hk], s["k_weight"])):
            y = y / (y.square().sum(-1, keepdim=True) / D + s["eps"]).sqrt() * w.double()
            z = torch.complex(y[..., first], y[..., second]) * turn
            y = y.clone()
            y[..., first], y[..., second] = z.real, z.imag
            parts.append(y)
        v = x[:, H + Hk:]
        at = s["table"][n].long()[p // page]
        kc[at, :, p % page], vc[at, :, p % page] = parts[1], v
        qs.append(parts[0]), ks.append(parts[1]), vs.append(v)
    dense = c["dense"]
    return dict(q=torch.cat(qs), k=torch.cat(ks) if dense else None, v=torch.cat(vs) if dense else None,
                k_cache=kc, v_cache=vc)


def _to_e4m3(y):
    """The nearest value with 4 significant bits, exponent -6 or more, at most 448; ties to even."""
    step = torch.exp2((torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3.0))
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def _least_scale(top):
    """Powers of two: for each value of top the first with top <= 448 s, found from above."""
    s = torch.full_like(top, 2.0 ** 130)
    while bool((fits := (top <= 224.0 * s) & (s > 2.0 ** -100)).any()):
        s = torch.where(fits, s / 2, s)
    return s


def _exact_append8(s):
    c = s["case"]
    page = c["page"]
    cu, kv, table = s["cu"].tolist(), s["kv_lens"].tolist(), s["table"].tolist()
    out = {x: s[x].double() for x in ("k_cache", "v_cache", "k_scale", "v_scale")}
    todo = []  # (page, first row of the block, rows held before, first new row, rows, first token)
    for n in range(c["N"]):
        a = kv[n] - (cu[n + 1] - cu[n])
        while a < kv[n]:
            b = min(a // BLOCK * BLOCK + BLOCK, kv[n])
            todo.append((table[n][a // page], a // BLOCK * BLOCK % page, a % BLOCK, b - a, cu[n] + a - kv[n] + cu[n + 1] - cu[n]))
            a = b
    if len(todo) > 6000:
        return None
    for x in ("k", "v"):
        cache, scale = out[x + "_cache"], out[x + "_scale"]
        tops = torch.stack([s[x][t:t + r].double().abs().amax((0, 2)) for _, _, _, r, t in todo])
        fits = _least_scale(tops)
        for (pg, row, held, r, t), fit in zip(todo, fits):
            old = scale[pg, :, row // BLOCK].clone()
            grown = torch.maximum(fit, old) if held else fit
            scale[pg, :, row // BLOCK] = grown
            if held:
                cache[pg, :, row:row + held] = _to_e4m3(cache[pg, :, row:row + held] * (old / grown)[:, None, None])
            cache[pg, :, row + held:row + held + r] = _to_e4m3(s[x][t:t + r].double().transpose(0, 1) / grown[:, None, None])
    return out


def _exact_rows(s, x, n, length):
    """Sequence n's keys or values, [length, Hk, D]."""
    page = s["case"]["page"]
    pages = s["table"][n, :-(-length // page)].long()
    if x + "_scale" not in s:
        rows = s[x + "_cache"][pages].double()
    else:
        held = s[x + "_cache"].view(torch.uint8)[pages].view(torch.float8_e4m3fn).double()
        p, h, m, d = held.shape
        rows = (held.view(p, h, m // BLOCK, BLOCK, d) * s[x + "_scale"][pages].double()[..., None, None]).view(p, h, m, d)
    return rows.transpose(1, 2).reshape(-1, rows.shape[1], rows.shape[3])[:length]


def _exact_decode(s):
    c, q = s["case"], s["q"]
    N, nq, H, Hk, D, page = c["N"], c["nq"], c["H"], c["Hk"], c["D"], c["page"]
    rows = q.view(N, nq, Hk, H // Hk, D).double()
    out = torch.empty_like(rows)
    weights = s["weights"].double() if "weights" in s else None
    for n, length in enumerate(s["kv_lens"].tolist()):
        k, v = _exact_rows(s, "k", n, length), _exact_rows(s, "v", n, length)
        scores = torch.einsum("ihgd,jhd->ihgj", rows[n], k) / math.sqrt(D)
        last = torch.arange(length - nq, length, device=q.device)
        unseen = torch.arange(length, device=q.device)[None, :] > last[:, None]
        w = torch.softmax(scores.masked_fill(unseen[:, None, None, :], float("-inf")), -1)
        out[n] = torch.einsum("ihgj,jhd->ihgd", w, v)
        if weights is not None:
            gain = w.sum((0, 2))  # [Hk, length]
            for a in range(0, length, page):
                pg, b = int(s["table"][n, a // page]), min(a + page, length)
                fresh = torch.arange(a, b, device=q.device) >= length - nq
                weights[pg, :, :b - a] = torch.where(fresh, 0.0, weights[pg, :, :b - a]) + gain[:, a:b]
    return dict(out=out.view(q.shape), weights=weights)


def _exact_prompt(s):
    c, q, k, cu = s["case"], s["q"], s["k"], s["cu"].tolist()
    T, H, D = q.shape
    Hk, page = k.shape[1], c["page"]
    weights = s["weights"].double()
    for n, (b, e) in enumerate(zip(cu[:-1], cu[1:])):
        gain = torch.zeros(e - b, Hk, dtype=torch.float64, device=q.device)
        begin = max(b, e - c["window"]) if c["window"] else b
        for h in range(H):
            kh = k[b:e, h // (H // Hk)].double()
            for r in range(begin, e, 2048):
                z = min(r + 2048, e)
                x = torch.einsum("id,jd->ij", q[r:z, h].double(), kh) / math.sqrt(D)
                i, j = torch.arange(r - b, z - b, device=q.device), torch.arange(e - b, device=q.device)
                w = torch.exp(x - s["lse"][r:z, h, None].double())
                gain[:, h // (H // Hk)] += torch.where(j[None, :] <= i[:, None], w, 0.0).sum(0)
        j = torch.arange(e - b, device=q.device)
        weights[s["table"][n].long()[j // page], :, j % page] = gain
    return weights


def _exact_evict(s):
    c = s["case"]
    page, keep, recent = c["page"], c["keep"], c["recent"]
    N, Hk, lens = c["N"], c["Hk"], s["kv_lens"].tolist()
    eight = "k_scale" in s
    names = ("k_cache", "v_cache", "weights") + (("k_scale", "v_scale") if eight else ())
    old = {x: s[x].double() for x in names}
    out = {x: old[x].clone() for x in names}
    kept = torch.full((N, Hk, keep), -1, dtype=torch.int32)
    rows = s["weights"].cpu()
    for n in range(N):
        table, new = s["table"][n].cpu().long(), s["new_table"][n].cpu().long()
        for h in range(Hk):
            j = torch.arange(lens[n])
            got = j
            if lens[n] > keep:
                w = rows[table[j // page], h, j % page]
                free = lens[n] - recent
                best = sorted(range(free), key=lambda i, w=w.tolist(): (-w[i], i))[:keep - recent]
                got = torch.cat([torch.tensor(sorted(best), dtype=torch.long), torch.arange(free, lens[n])])
            m = got.numel()
            kept[n, h, :m] = got.int()
            i = torch.arange(m)
            a, ar, b, br = table[got // page], got % page, new[i // page], i % page
            out["weights"][b, h, br] = old["weights"][a, h, ar]
            for x in ("k", "v"):
                held = old[x + "_cache"][a, h, ar]
                if eight:
                    scale = old[x + "_scale"][a, h, ar // BLOCK]
                    most = torch.stack([t.max() for t in scale.split(BLOCK)])
                    out[x + "_scale"][b[::BLOCK], h, br[::BLOCK] // BLOCK] = most
                    held = _to_e4m3(held * (scale / most.repeat_interleave(BLOCK)[:m])[:, None])
                out[x + "_cache"][b, h, br] = held
    return dict(lens=torch.tensor([min(x, keep) for x in lens], dtype=torch.int32), kept=kept,
                **{x: out.get(x) for x in ("k_cache", "v_cache", "k_scale", "v_scale", "weights")})
