"""GPU: what precision the shared-prefix decode's outputs have, by their type, the
queries' and the rows of a KV head (bounds as in test_gpu_prefix_decode).

A query row is a pair of fp16 terms (d = 2^-19 D) unless queries and outputs are bf16 and
more than 128 rows share a prefix; there it is rounded to fp16 once (d = 2^-11 D, an
eighth of what bf16 queries carry already). Weights are pairs for fp16 and fp32 outputs
(e = 2^-22), rounded once for bf16 (e = 2^-11, an eighth of the output's own rounding)."""
import numpy as np
import pytest
import torch

import synth
from test_gpu_prefix_decode import DEV, U, Setup, contiguous

pytestmark = pytest.mark.gpu


def _cases(seed, rows, q_dtype, scale, pre=300, n_kv=1):
    """Queries of `rows` rows per KV head behind one prefix, with a few own tokens."""
    S = Setup(seed, n_kv, 4, 4)
    G = max(g for g in range(1, 17) if rows % g == 0)
    B = rows // G
    own = [(7 * i) % 40 for i in range(B)]
    pd, od = S.tokens(pre), [S.tokens(n) for n in own]
    q = torch.from_numpy(scale * S.rng.standard_normal((B, n_kv * G, 128))).to(q_dtype)
    P, Q = contiguous(S, [pre], [pd]), contiguous(S, own, od)
    heads = S.heads(*pd), [S.heads(*x) for x in od]
    return S, G, P, Q, q, heads


def _rows(S, G, q, heads):
    """(b, head, fp64 output, A, B, D, tokens) of every query row: A = sum_t p_t |v_hat_t|
    by coordinate, B = sum_t p_t times the norm of v_hat_t."""
    pre, own = heads
    for b in range(q.shape[0]):
        for h in range(S.n_kv):
            k, v = (np.concatenate([pre[h][i], own[b][h][i]]) for i in (0, 1))
            for g in range(h * G, (h + 1) * G):
                x = q[b, g].double().numpy()
                s = k @ x / np.sqrt(128)
                p = np.exp(s - s.max())
                p /= p.sum()
                D = (np.abs(k) @ np.abs(x)).max() / np.sqrt(128)
                yield b, g, p @ v, p @ np.abs(v), p @ np.linalg.norm(v, axis=1), D, len(k)


@pytest.mark.parametrize("q_dtype,rows", [
    (torch.bfloat16, 1), (torch.bfloat16, 16), (torch.bfloat16, 64), (torch.bfloat16, 65),
    (torch.bfloat16, 112), (torch.bfloat16, 128), (torch.float16, 16), (torch.float32, 128),
    (torch.float32, 129), (torch.float16, 256), (torch.float32, 330)])
def test_bf16_outputs_of_query_pairs(q_dtype, rows):
    """Sharp logits, so that what a query row loses shows: an output is bf16's half step
    from the exact one, and its weights' rounding.

    Where one token takes all, A can be next to 0 in a coordinate, and the fp32 sums in
    the rotated domain count: O_j = sum_t P_t c_tj takes n / 16 additions (16 tokens to a
    step of the products), at most 16 for the merge of its records and 7 in the inverse
    rotation, each good to 2^-23 of sum_t P_t |c_tj|. The inverse rotation adds 128 of
    them over 128: (1 / 128) sum_j |c_tj| <= |c_t| / sqrt(128), the norm of v_hat_t over
    its stored norm, so a coordinate is off by at most (n / 16 + 23) 2^-23 B."""
    S, G, P, Q, q, heads = _cases(71, rows, q_dtype, 40.0)
    out = torch.empty(q.shape, dtype=torch.bfloat16, device=DEV)
    gs = torch.tensor([0, q.shape[0]], dtype=torch.int32, device=DEV)
    got = Q.decode_prefix(q.to(DEV), P, gs, out=out).double().cpu().numpy()
    assert Q.flags() == 0
    for b, g, ref, A, B, D, n in _rows(S, G, q, heads):
        e = 2.0 ** -11 + n * 2.0 ** -26 + 2.0 ** -15
        tol = U[torch.bfloat16] * np.abs(ref) + (np.expm1(2 * 2.0 ** -19 * D) + e) * A + \
            (n / 16 + 23) * 2.0 ** -23 * B
        err = np.abs(got[b, g] - ref)
        assert np.all(err <= tol), (b, g, (err / tol).max())


@pytest.mark.parametrize("rows", [1, 16, 64, 65, 128, 129, 300])
def test_fp32_outputs(rows):
    """fp32 outputs, ordinary logits and value norms: 2e-6 of the output's norm. What is
    left are independent roundings: each weight's 2^-22 (its logit: 22-bit pairs, an fp32
    sum of 8 steps, a scaling of a logit below 8; its exponential, 2^-22; its own pair),
    at most 2^-20 in all with logits of magnitude 8, which add as their root over a row's
    effective tokens like the output itself does: 2^-20 = 1e-6 of its norm, and as much
    again for the sums."""
    S, G, P, Q, q, heads = _cases(72, rows, torch.float32, 1.0, pre=700, n_kv=2)
    gs = torch.tensor([0, q.shape[0]], dtype=torch.int32, device=DEV)
    got = Q.decode_prefix(q.to(DEV), P, gs).double().cpu().numpy()
    assert Q.flags() == 0
    num = den = 0.0
    for b, g, ref, *_ in _rows(S, G, q, heads):
        num += np.sum((got[b, g] - ref) ** 2)
        den += np.sum(ref ** 2)
    assert np.sqrt(num / den) <= 2e-6, np.sqrt(num / den)


@pytest.mark.parametrize("lead,n", [(7.6, 2000), (4.0, 55), (10.0, 20000)])
def test_logits_are_not_shrunk(lead, n):
    """One heavy token against n - 1 light ones of about the same weight together, their
    values orthogonal: the ratio of the two parts of an fp32 output is the heavy
    logit's, whatever the sums of values lose in common.

    The mean of its error over 64 rows is what the products lose to truncation: a step
    at most 2^-23 of the sum so far. With the small terms first (low parts, then the
    blocks by energy) the sums before the last step are together at most the logit s
    itself, so 2 * 2^-23 s; the remaining roundings (2^-22 s each, either sign) average
    to an eighth of that, twice over; 2^-22 (s + 2) in all."""
    S = Setup(73, 1, 4, 4)
    sig = np.sqrt(np.concatenate([S.E[0], S.E[0]]) / 2)
    sig /= np.linalg.norm(sig)
    u = S.rng.standard_normal(128) * sig
    u /= np.linalg.norm(u)
    k = 0.02 * S.rng.standard_normal((n, 128)) * sig
    k[0] = lead * u
    a, b = S.rng.standard_normal((2, 128))
    b -= a * (a @ b) / (a @ a)
    v = np.tile(b, (n, 1))
    v[0] = a
    data = synth.to_bf16_bits(k[:, None]), synth.to_bf16_bits(v[:, None])
    q = np.sqrt(128) * u * (1 + 0.1 * S.rng.standard_normal((4, 16, 1)))
    q = torch.from_numpy(q + 0.1 * S.rng.standard_normal((4, 16, 128))).float()
    P, Q = contiguous(S, [n], [data]), contiguous(S, [0] * 4, [([], [])] * 4, extra=8)
    gs = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    got = Q.decode_prefix(q.to(DEV), P, gs).double().cpu().numpy()
    kh, vh = S.heads(*data)[0]
    parts = np.linalg.pinv(np.stack([vh[0], vh[1]], axis=1))
    errs, s0 = [], []
    for x, o in zip(q.double().numpy().reshape(-1, 128), got.reshape(-1, 128)):
        s = kh @ x / np.sqrt(128)
        heavy, light = parts @ o
        errs.append(np.log(heavy / light) - (s[0] - np.log(np.exp(s[1:]).sum())))
        s0.append(s[0])
    assert abs(np.mean(errs)) <= 2.0 ** -22 * (np.mean(s0) + 2), (np.mean(errs), np.mean(s0))
