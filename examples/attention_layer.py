"""The softmax-attention layers of a hybrid stack, as a serving loop runs them: a batch of
requests that share a document, the document's prompt once, each request's own prompt on top
of it, then decode steps; keys and values in a paged cache throughout. Every output is
compared with one long prompt through gdn_attn_prefill.

    python examples/attention_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gated_delta_rule_chunk_gb300 import binding as B  # noqa: E402
from gated_delta_rule_chunk_gb300 import rope_table  # noqa: E402


def main(requests=6, document=512, own=37, steps=4, H=16, Hk=2, D=128, page=64, seed=0) -> float:
    """Returns the largest difference from the one-prompt result."""
    torch.manual_seed(seed)
    dev = torch.device("cuda")
    width = (H + 2 * Hk) * D
    doc = torch.randn(document, width, device=dev, dtype=torch.bfloat16)
    ask = torch.randn(requests, own + steps, width, device=dev, dtype=torch.bfloat16)
    layer = dict(H=H, Hk=Hk, D=D, q_weight=torch.ones(D, device=dev),
                 k_weight=torch.ones(D, device=dev), rope=rope_table(4096, D // 4, device=dev))

    # The cache: the document's pages are the first columns of every request's row.
    shared = document // page * page
    per = -(-(document + own + steps) // page) - shared // page
    n_pages = shared // page + requests * per
    kc, vc = (torch.zeros(n_pages, Hk, page, D, device=dev, dtype=torch.bfloat16) for _ in range(2))
    table = torch.empty(requests, shared // page + per, dtype=torch.int32, device=dev)
    table[:, :shared // page] = torch.arange(shared // page, device=dev)
    table[:, shared // page:] = shared // page + torch.arange(requests * per, device=dev).view(requests, per)
    lens = torch.full((requests,), document, dtype=torch.int32, device=dev)

    # The document's prompt, appended once.
    B.gdn_attn_front(doc[:shared], page_table=table[:1].contiguous(), k_cache=kc, v_cache=vc,
                     output_kv=False, **layer)

    # Each request's tokens: the prompt as one verify-like step of `own` tokens, then one by
    # one. What of the document does not fill a page belongs to each request.
    rest = torch.cat([doc[shared:].expand(requests, -1, -1), ask], 1)
    lens.fill_(shared)
    got, at = [], 0
    for n in [rest.shape[1] - steps] + [1] * steps:
        x = rest[:, at:at + n].reshape(-1, width).contiguous()
        at += n
        lens += n
        cu = torch.arange(requests + 1, dtype=torch.int32, device=dev) * n
        q, _, _ = B.gdn_attn_front(x, cu_seqlens=cu, kv_lens=lens, page_table=table, k_cache=kc,
                                   v_cache=vc, output_kv=False, **layer)
        q = q.view(requests, n, H, D)
        for b in range(0, n, 64 * Hk // H):  # at most 64 rows a key head in a call
            e = min(b + 64 * Hk // H, n)
            got.append(B.gdn_attn_decode(q[:, b:e].contiguous(), kc, vc, table, lens - (n - e), shared,
                                         out_dtype=torch.float32))
    got = torch.cat(got, 1)

    # The same as one packed batch of long prompts.
    x = torch.cat([torch.cat([doc, a]) for a in ask])
    each = document + own + steps
    cu = torch.arange(requests + 1, dtype=torch.int32, device=dev) * each
    q, k, v = B.gdn_attn_front(x, cu_seqlens=cu, **layer)
    want = B.gdn_attn_prefill(q, k, v, cu, out_dtype=torch.float32).view(requests, each, H, D)
    return (got - want[:, shared:]).abs().max().item()


if __name__ == "__main__":
    print(f"largest difference between the cached steps and one prompt: {main():.2e}")
