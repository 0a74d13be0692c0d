"""The softmax-attention layer's operators as workloads: the front end (q/k norm, rotary
positions, append to the paged cache), causal attention over packed prompts, and decode
attention over the paged cache with an optional prefix that all sequences share.

`run` computes an operator in its plain form (elementary torch operations in 32 bits, one
rounding at the end) or, where `own` is true, through the package's entry points. `exact`
evaluates the definitions in 64 bits.
"""
import math
import random

import torch

own = False

PAGE_SIZES = (16, 32, 64, 128, 256)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # One token of one conversation entering its layer: nothing but latency.
        dict(name="front_step_1", op="front", N=1, lo=1, hi=1, past=8190, H=16, Hk=2, D=128, rot=64,
             interleaved=False, page=16, x="bf16", out="bf16", dense=False, lens_seed=1),
        # A decode step of a full batch, every sequence at a position of its own.
        dict(name="front_step_64", op="front", N=64, lo=1, hi=1, past=8190, H=32, Hk=8, D=128, rot=128,
             interleaved=False, page=64, x="bf16", out="bf16", dense=False, lens_seed=2),
        # A whole prompt; a quarter of the head rotated; k and v kept dense for the prompt's own
        # attention and appended to the cache.
        dict(name="front_prompt_4096", op="front", N=1, lo=4096, hi=4096, past=0, H=16, Hk=2, D=128,
             rot=32, interleaved=False, page=64, x="bf16", out="bf16", dense=True, lens_seed=3),
        # Several prompts of odd lengths that go on from what the cache holds; 32-bit projection
        # output and results, interleaved pairs, head size 64.
        dict(name="front_ragged_f32", op="front", N=8, lo=1, hi=2048, past=777, H=32, Hk=4, D=64,
             rot=64, interleaved=True, page=32, x="f32", out="f32", dense=True, lens_seed=4),
        # A batch of short questions: many sequences, most shorter than a tile.
        dict(name="prefill_short_20", op="prefill", N=20, lo=1, hi=204, H=16, Hk=4, D=128, lens_seed=5),
        # The prompt length of the delta-rule workloads.
        dict(name="prefill_4096", op="prefill", N=1, lo=4096, hi=4096, H=16, Hk=4, D=128, lens_seed=6),
        # Packed prompts of uneven lengths.
        dict(name="prefill_ragged_8", op="prefill", N=8, lo=1, hi=2048, H=32, Hk=8, D=128, lens_seed=7),
        # Head size 64, a key head for every query head, an odd length.
        dict(name="prefill_4001_d64", op="prefill", N=1, lo=4001, hi=4001, H=16, Hk=16, D=64, lens_seed=8),
        # A long document.
        dict(name="prefill_16384", op="prefill", N=1, lo=16384, hi=16384, H=32, Hk=8, D=128, lens_seed=9),
        # One conversation's next token over its own context: latency and one long axis to split.
        dict(name="decode_1", op="decode", N=1, nq=1, lo=8191, hi=8191, shared=0, H=16, Hk=4, D=128,
             page=16, lens_seed=10),
        # A batch's next tokens, contexts of very different lengths.
        dict(name="decode_64", op="decode", N=64, nq=1, lo=1, hi=8192, shared=0, H=32, Hk=8, D=128,
             page=64, lens_seed=11),
        # A batch that shares a long document, each sequence with a conversation of its own.
        dict(name="decode_shared_64", op="decode", N=64, nq=1, lo=1, hi=1024, shared=16384, H=32, Hk=8,
             D=128, page=16, lens_seed=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("front", "prefill", "decode"))
    while True:
        Hk = rng.choice((1, 2, 3, 4, 8))
        G = rng.choice((1, 2, 3, 4, 5, 6, 7, 8, 16))
        D = rng.choice((64, 128, 128))
        if Hk * G * D == 24 * 128 or Hk * (G + 2) * D == 24 * 128:  # row widths of no model here
            continue
        c = dict(op=op, H=Hk * G, Hk=Hk, D=D, lens_seed=rng.randrange(1 << 20))
        if op == "front":
            step = rng.random() < 0.4
            N = _log(rng, 1, 256) if step else _log(rng, 1, 32)
            hi = 1 if step else _log(rng, 2, 8192)
            kinds = rng.choice((("bf16", "bf16"), ("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")))
            c.update(N=N, lo=1, hi=hi, past=rng.choice((0, _log(rng, 1, 16384))),
                     rot=rng.choice((16, 32, c["D"] // 2, c["D"])), interleaved=rng.random() < 0.5,
                     page=rng.choice(PAGE_SIZES), x=kinds[0], out=kinds[1], dense=not step)
            if N * hi <= 32768:
                return c
        elif op == "prefill":
            N, hi = _log(rng, 1, 32), _log(rng, 1, 16384)
            c.update(N=N, lo=max(1, hi // rng.choice((1, 2, 8, 1000000))), hi=hi)
            if N * hi * hi * c["H"] <= 16384 * 16384 * 16 and N * hi <= 65536:
                return c
        else:
            N, hi = _log(rng, 1, 128), _log(rng, 1, 16384)
            page = rng.choice(PAGE_SIZES)
            shared = rng.choice((0, 0, 1, 1, 1)) * (_log(rng, page, 32768) // page * page)
            nq = rng.choice((1, 1, 1, 2, 3, 5, 8))
            c.update(N=N, nq=nq, lo=max(nq, hi // rng.choice((1, 2, 1000000))), hi=max(nq, hi),
                     shared=shared, page=page)
            if (nq * G <= 64 and N * c["hi"] * Hk <= 1 << 22
                    and N * nq * c["H"] * (shared + c["hi"]) <= 1 << 28):
                return c


def _lens(case):
    r = random.Random(case["lens_seed"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["N"])]


def _esz(kind):
    return 4 if kind == "f32" else 2


def work(case):
    H, Hk, D, lens = case["H"], case["Hk"], case["D"], _lens(case)
    T = sum(lens)
    if case["op"] == "front":
        ein, eout = _esz(case["x"]), _esz(case["out"])
        kv = 2 * T * Hk * D * eout
        table = 4 * case["rot"] * min(T, case["past"] + max(lens))  # each position's row once
        return {"bytes": T * (H + 2 * Hk) * D * ein + T * H * D * eout + kv * (2 if case["dense"] else 1)
                + table, "flops": 8 * T * (H + Hk) * D}
    if case["op"] == "prefill":
        return {"bytes": 2 * T * (2 * H + 2 * Hk) * D,
                "flops": 4 * D * H * sum(n * (n + 1) // 2 for n in lens)}
    N, nq, S = case["N"], case["nq"], case["shared"]
    pairs = sum(nq * (S + n) - nq * (nq - 1) // 2 for n in lens)
    return {"bytes": 4 * Hk * D * (S + T) + 4 * N * nq * H * D, "flops": 4 * D * H * pairs}


# ---------------------------------------------------------------- inputs
def _pages(g, N, counts, shared_pages):
    """A page table [N, width] of physical pages in scattered order; the first shared_pages
    entries of every row are the same pages. Returns it and the number of pages."""
    width = shared_pages + max(counts)
    n_pages = shared_pages + sum(counts)
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    count = torch.tensor(counts, device="cuda")
    first = shared_pages + torch.cumsum(count, 0) - count
    i = torch.arange(width, device="cuda")[None, :]
    own_page = first[:, None] + torch.minimum((i - shared_pages).clamp(min=0), (count - 1)[:, None])
    return perm[torch.where(i < shared_pages, i, own_page)].contiguous(), n_pages


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    H, Hk, D, N, lens = case["H"], case["Hk"], case["D"], case["N"], _lens(case)
    T = sum(lens)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)

    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    if case["op"] == "prefill":
        return dict(case=case, q=normal(T, H, D), k=normal(T, Hk, D), v=normal(T, Hk, D), cu=cu,
                    longest=max(lens))
    page = case["page"]
    if case["op"] == "decode":
        S = case["shared"]
        table, n_pages = _pages(g, N, [-(-n // page) for n in lens], S // page)
        shape = (N, H, D) if case["nq"] == 1 else (N, case["nq"], H, D)
        return dict(case=case, q=normal(*shape), k_cache=normal(n_pages, Hk, page, D),
                    v_cache=normal(n_pages, Hk, page, D), table=table,
                    kv_lens=torch.tensor([S + n for n in lens], device="cuda", dtype=torch.int32))
    xt, ot = (torch.float32 if case[k] == "f32" else torch.bfloat16 for k in ("x", "out"))
    kv = [case["past"] + n for n in lens]
    table, n_pages = _pages(g, N, [-(-n // page) for n in kv], 0)
    rot = case["rot"]
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    angle = torch.arange(max(kv), device="cuda", dtype=torch.float64)[:, None] * freq
    return dict(case=case, x=normal(T, (H + 2 * Hk) * D, dtype=xt) * 2.0, cu=cu,
                kv_lens=torch.tensor(kv, device="cuda", dtype=torch.int32), table=table,
                k_cache=normal(n_pages, Hk, page, D, dtype=ot),
                v_cache=normal(n_pages, Hk, page, D, dtype=ot),
                q_weight=1.0 + 0.1 * normal(D, dtype=torch.float32),
                k_weight=1.0 + 0.1 * normal(D, dtype=torch.float32),
                rope=torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32), eps=1e-6)


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
                               output_kv=c["dense"], out_dtype=s["k_cache"].dtype)
    return dict(q=q, k=k, v=v, k_cache=s["k_cache"], v_cache=s["v_cache"])


def _own_prefill(s):
    from gated_delta_rule_chunk_gb300 import binding as B
    return B.gdn_attn_prefill(s["q"], s["k"], s["v"], cu_seqlens=s["cu"])


def _own_decode(s):
    from gated_delta_rule_chunk_gb300 import binding as B
    return B.gdn_attn_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"],
                             shared_len=s["case"]["shared"])


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


def _plain_front(s):
    c = s["case"]
    H, Hk, D, page = c["H"], c["Hk"], c["D"], c["page"]
    x = s["x"].float()
    T = x.shape[0]
    dt = s["k_cache"].dtype
    t = torch.arange(T, device=x.device)
    n = torch.searchsorted(s["cu"][1:], t, right=True)
    pos = (s["kv_lens"] - s["cu"][1:])[n] + t  # the sequence's new tokens are its last ones
    cos, sin = s["rope"][pos].chunk(2, 1)
    q, k, v = (y.view(T, -1, D) for y in x.split([H * D, Hk * D, Hk * D], 1))
    q = _norm_rotate(q, s["q_weight"], s["eps"], cos, sin, c["interleaved"]).to(dt)
    k = _norm_rotate(k, s["k_weight"], s["eps"], cos, sin, c["interleaved"]).to(dt)
    v = v.to(dt)
    at = s["table"][n, pos // page].long()
    s["k_cache"][at, :, pos % page] = k
    s["v_cache"][at, :, pos % page] = v
    return dict(q=q, k=k if c["dense"] else None, v=v if c["dense"] else None, k_cache=s["k_cache"],
                v_cache=s["v_cache"])


def _weigh(scores, seen):
    """exp(scores - row maximum) where `seen` (in place), and the row sums."""
    scores.masked_fill_(~seen, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    scores.sub_(torch.where(top > float("-inf"), top, 0.0)).exp_()
    return scores, scores.sum(-1, keepdim=True)


def _plain_prefill(s):
    q, k, v, cu, L = s["q"], s["k"], s["v"], s["cu"].long(), s["longest"]
    T, H, D = q.shape
    Hk, N = k.shape[1], cu.numel() - 1
    t = torch.arange(T, device=q.device)
    n = torch.searchsorted(cu[1:], t, right=True)
    i = t - cu[n]

    def padded(x):  # [T, heads, D] -> [N, heads, L, D] in 32 bits
        y = x.new_zeros(N, L, x.shape[1], D, dtype=torch.float32)
        y[n, i] = x.float()
        return y.transpose(1, 2)

    qp, kp, vp = padded(q) * D ** -0.5, padded(k), padded(v)
    rows = qp.reshape(N, Hk, H // Hk * L, D)
    scores = (rows @ kp.transpose(-1, -2)).view(N, Hk, H // Hk, L, L)
    a = torch.arange(L, device=q.device)
    p, total = _weigh(scores, a[None, :] <= a[:, None])
    out = (p.view(N, Hk, -1, L) @ vp).view(N, H, L, D) / total.view(N, H, L, 1)
    return out[n, :, i].to(q.dtype)


def _plain_decode(s):
    c, q = s["case"], s["q"]
    N, nq, H, Hk, D, S, page = c["N"], c["nq"], c["H"], c["Hk"], c["D"], c["shared"], c["page"]
    G = H // Hk
    rows = (q.float() * D ** -0.5).view(N, nq, Hk, G, D).permute(2, 0, 3, 1, 4)  # [Hk, N, G, nq, D]
    pre, own_pages = s["table"][0, :S // page].long(), s["table"][:, S // page:].long()
    kp, vp = (x[pre].float().transpose(0, 1).reshape(Hk, S, D) for x in (s["k_cache"], s["v_cache"]))
    ko, vo = (x[own_pages].float().permute(2, 0, 1, 3, 4).reshape(Hk, N, -1, D)
              for x in (s["k_cache"], s["v_cache"]))
    shared = (rows.reshape(Hk, N * G * nq, D) @ kp.transpose(-1, -2)).view(Hk, N, G * nq, S)
    apart = rows.reshape(Hk, N, G * nq, D) @ ko.transpose(-1, -2)
    scores = torch.cat([shared, apart], -1).view(Hk, N, G, nq, -1)
    j = torch.arange(scores.shape[-1], device=q.device)
    last = s["kv_lens"].long()[:, None] - nq + torch.arange(nq, device=q.device)  # [N, nq]
    p, total = _weigh(scores, j <= last[None, :, None, :, None])
    p = p.view(Hk, N, G * nq, -1)
    out = (p[..., :S].reshape(Hk, N * G * nq, S) @ vp).view(Hk, N, G * nq, D) + p[..., S:] @ vo
    total = total.view(Hk, N, G * nq, 1)
    out = torch.where(total > 0, out / total, 0.0).view(Hk, N, G, nq, D)
    return out.permute(1, 3, 0, 2, 4).reshape(q.shape).to(q.dtype)


_own = dict(front=_own_front, prefill=_own_prefill, decode=_own_decode)
_plain = dict(front=_plain_front, prefill=_plain_prefill, decode=_plain_decode)


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return dict(front=_exact_front, prefill=_exact_prefill, decode=_exact_decode)[case["op"]](s)


def _exact_front(s):
    c = s["case"]
    H, Hk, D, page, rot = c["H"], c["Hk"], c["D"], c["page"], c["rot"]
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    qs, ks, vs = [], [], []
    cu, kv = s["cu"].tolist(), s["kv_lens"].tolist()
    first = torch.arange(0, rot, 2) if c["interleaved"] else torch.arange(rot // 2)
    second = first + (1 if c["interleaved"] else rot // 2)
    for n in range(c["N"]):
        x = s["x"][cu[n]:cu[n + 1]].double().view(-1, H + 2 * Hk, D)
        p = torch.arange(kv[n] - x.shape[0], kv[n], device=x.device)
        turn = torch.complex(s["rope"][p, :rot // 2].double(), s["rope"][p, rot // 2:].double())[:, None, :]
        parts = []
        for y, w in ((x[:, :H], s["q_weight"]), (x[:, H:H + Hk], s["k_weight"])):
            y = y / (y.square().sum(-1, keepdim=True) / D + s["eps"]).sqrt() * w.double()
            z = torch.complex(y[..., first], y[..., second]) * turn
            y = y.clone()
            y[..., first], y[..., second] = z.real, z.imag
            parts.append(y)
        v = x[:, H + Hk:]
        where = s["table"][n].long()[p // page]
        kc[where, :, p % page], vc[where, :, p % page] = parts[1], v
        qs.append(parts[0]), ks.append(parts[1]), vs.append(v)
    dense = c["dense"]
    return dict(q=torch.cat(qs), k=torch.cat(ks) if dense else None, v=torch.cat(vs) if dense else None,
                k_cache=kc, v_cache=vc)


def _exact_attend(q, k, v, last):
    """q [r, D], k, v [n, D], row i sees keys 0 .. last[i]; in 64 bits."""
    D = q.shape[-1]
    scores = torch.einsum("rd,nd->rn", q.double(), k.double()) / math.sqrt(D)
    unseen = torch.arange(k.shape[0], device=q.device)[None, :] > last[:, None]
    weights = torch.softmax(scores.masked_fill(unseen, float("-inf")), -1)
    return torch.einsum("rn,nd->rd", weights, v.double())


def _exact_prefill(s):
    q, k, v, cu = s["q"], s["k"], s["v"], s["cu"].tolist()
    G = q.shape[1] // k.shape[1]
    out = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    for b, e in zip(cu[:-1], cu[1:]):
        for h in range(q.shape[1]):
            for r in range(b, e, 2048):
                z = min(r + 2048, e)
                out[r:z, h] = _exact_attend(q[r:z, h], k[b:z, h // G], v[b:z, h // G],
                                            torch.arange(r - b, z - b, device=q.device))
    return out


def _exact_decode(s):
    c, q = s["case"], s["q"]
    N, nq, H, Hk, D, page = c["N"], c["nq"], c["H"], c["Hk"], c["D"], c["page"]
    G = H // Hk
    rows = q.view(N, nq, Hk, G, D)
    out = torch.empty(rows.shape, dtype=torch.float64, device=q.device)
    for n, length in enumerate(s["kv_lens"].tolist()):
        pages = s["table"][n, :-(-length // page)].long()
        k, v = s["k_cache"][pages], s["v_cache"][pages]  # [pages, Hk, page, D]
        last = torch.arange(length - nq, length, device=q.device).repeat_interleave(G)
        for h in range(Hk):
            got = _exact_attend(rows[n, :, h].reshape(nq * G, D), k[:, h].reshape(-1, D)[:length],
                                v[:, h].reshape(-1, D)[:length], last)
            out[n, :, h] = got.view(nq, G, D)
    return out.view(q.shape)
