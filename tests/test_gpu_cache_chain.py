"""The operators on a paged cache as a hybrid model's layers run them: a prompt of
several sessions behind a shared prefix, then single tokens out of a captured
graph, the attention layer beside a delta-rule layer.

The attention over everything that was appended is held to the 64-bit definition
over the rows that the same norm and rotation give: what append rounds once is the
reference's input, so the bounds are those of the attention's own tests."""
import pytest
import torch

from cache_ref import DEV, attention_ref, rotate_ref
from layer_ref import HALF, U, offsets
from parity import say

import gated_delta_rule_81_amd as kda

H, HQ, D, PAGE, SHARED = 2, 8, 128, 16, 70


def rope(rows, rot):
    a = torch.arange(rows, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return torch.cat([a.cos(), a.sin()], -1).float()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=str)
def test_prompt_then_tokens(dtype):
    g = torch.Generator().manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype).to(DEV)
    prompt, steps, N = [37, 1, 20], 4, 3
    table = rope(300, 64).to(DEV)
    pages = torch.randperm(40, generator=g).int().to(DEV)
    prefix, own = pages[:5].contiguous(), pages[5:26].reshape(N, 7).contiguous()
    kc, vc = (torch.full((40, PAGE, H, D), float("nan"), dtype=dtype, device=DEV) for _ in range(2))
    plen = torch.tensor([SHARED], dtype=torch.int32, device=DEV)
    one = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    say("cache chain", dtype)

    # the shared text is one session's prompt, whose pages the others then read
    ks, vs = r(SHARED, H, D), r(SHARED, H, D)
    kda.cache_append(ks, vs, kc, vc, prefix[None], plen, table=table,
                     positions=torch.arange(SHARED, dtype=torch.int32, device=DEV))

    # a prompt: norm of q and k, rotation and append, attention; a delta-rule layer beside it
    cu, lens = offsets(prompt).to(DEV), one(*prompt)
    T = sum(prompt)
    where = torch.cat([torch.arange(n) for n in prompt]).int().to(DEV) + SHARED
    q, k, v = r(T, HQ, D), r(T, H, D), r(T, H, D)
    qn, kn = kda.qk_norm(q, k, kind="rms")
    qr = kda.cache_append(kn, v, kc, vc, own, lens, cu, q=qn, table=table, positions=where)
    out, _ = kda.prefix_attention(qr, kc, vc, own, lens, prefix, plen, cu, output_lse=True)
    gates = lambda *s: (-torch.rand(*s, generator=g)).to(DEV)
    _, state = kda.chunk_fwd(*(x[None] for x in kda.qk_norm(out, out.clone())), out[None],
                             gates(1, T, HQ, D), gates(1, T, HQ).neg(), None, cu)
    assert torch.isfinite(state).all()

    # single tokens, captured once: lengths and positions move on by themselves
    tok = dict(q=r(N, HQ, D), k=r(N, H, D), v=r(N, H, D))
    la, beta = gates(N, HQ, D), gates(N, HQ).neg()
    at = lens + SHARED - 1

    def step():
        lens.add_(1), at.add_(1)
        a, b = kda.qk_norm(tok["q"], tok["k"], kind="rms")
        a = kda.cache_append(b, tok["v"], kc, vc, own, lens, q=a, table=table, positions=at)
        y, _ = kda.prefix_attention(a, kc, vc, own, lens, prefix, plen)
        n, m = kda.qk_norm(y, y.clone())
        return a, b, y, kda.decode_step(n, m, y, la, beta, state)

    keep = [t.clone() for t in (lens, at, kc, vc, state)]
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for t, was in zip((lens, at, kc, vc, state), keep):
        t.copy_(was)
    rows_k = [[kn[cu[s] + i] for i in range(n)] for s, n in enumerate(prompt)]
    rows_v = [[v[cu[s] + i] for i in range(n)] for s, n in enumerate(prompt)]
    outs, queries = [], []
    for _ in range(steps):
        for t in tok.values():
            t.copy_(r(*t.shape))
        graph.replay()
        torch.cuda.synchronize()
        a, b, y, z = (t.clone() for t in got)
        assert torch.isfinite(z).all() and torch.isfinite(state).all()
        outs.append(y), queries.append(a)
        for s in range(N):
            rows_k[s].append(b[s]), rows_v[s].append(tok["v"][s].clone())
    assert lens.tolist() == [n + steps for n in prompt]

    # every key as it was rounded into the cache: within one rounding of the rotated rows
    host = lambda t: t.detach().cpu()
    total = [n + steps for n in prompt]
    for s in range(N):
        want = rotate_ref(torch.stack(rows_k[s]).double().cpu(), table.double().cpu(),
                          SHARED + torch.arange(total[s]), 0, False)
        have = torch.stack([kc[own[s, j // PAGE], j % PAGE] for j in range(total[s])]).double().cpu()
        assert ((have - want).abs() <= HALF[dtype] * want.abs() + 4 * U * want.abs().max()).all()
        vals = torch.stack([vc[own[s, j // PAGE], j % PAGE] for j in range(total[s])])
        assert torch.equal(vals, torch.stack(rows_v[s]))

    # the prompt's and each token's attention against the definition over the cache
    def check(y, query, lengths, new):
        ref, lse, wgt = attention_ref(host(query), host(kc), host(vc), host(own), torch.tensor(lengths),
                                      host(prefix), SHARED, new, D ** -0.5, D)
        A = float(query.double().norm(dim=-1).max() * kc.double().nan_to_num().norm(dim=-1).max()) * D ** -0.5
        rounded, n = HALF[dtype] if dtype == torch.bfloat16 else 0.0, SHARED + max(lengths)
        b = HALF[dtype] * ref.abs() + (rounded + (2 * (D + 8) * A + 2 * n + 100) * U) * wgt * (1 + HALF[dtype])
        assert ((y.double().cpu() - ref).abs() <= b).all()

    check(out, qr, prompt, prompt)
    for i in range(steps):
        check(outs[i], queries[i], [n + i + 1 for n in prompt], [1] * N)


@pytest.mark.gpu
def test_new_tokens_at_once_or_one_by_one():
    """Four drafts in one pass see what four single tokens see: the same rows in the cache, and
    attention within both passes' bounds of each other."""
    g = torch.Generator(device=DEV).manual_seed(3)
    r = lambda *s: torch.randn(*s, device=DEV, generator=g).bfloat16()
    N, n = 5, 4
    own = torch.arange(N * 4, dtype=torch.int32, device=DEV).reshape(N, 4)
    lens = torch.tensor([4, 9, 30, 64, 17], dtype=torch.int32, device=DEV)
    q, k, v = r(N, n, HQ, D), r(N, n, H, D), r(N, n, H, D)
    base_k, base_v = r(20, PAGE, H, D), r(20, PAGE, H, D)
    kc, vc = base_k.clone(), base_v.clone()
    say("drafts at once")
    flat = lambda t: t.flatten(0, 1)
    kda.cache_append(flat(k), flat(v), kc, vc, own, lens)
    a, la = kda.prefix_attention(flat(q), kc, vc, own, lens, output_lse=True)
    k2, v2 = base_k.clone(), base_v.clone()
    for i in range(n):
        now = lens - n + 1 + i
        kda.cache_append(k[:, i], v[:, i], k2, v2, own, now)
        b, lb = kda.prefix_attention(q[:, i].contiguous(), k2, v2, own, now, output_lse=True)
        torch.cuda.synchronize()
        # two passes' probabilities and outputs rounded once each, |v| under 6
        assert (a.view(N, n, HQ, D)[:, i].double() - b.double()).abs().max() <= 2 * 2 * HALF[torch.bfloat16] * 6
        assert torch.allclose(la.view(N, n, HQ)[:, i], lb, atol=1e-4)
    assert torch.equal(kc, k2) and torch.equal(vc, v2)
