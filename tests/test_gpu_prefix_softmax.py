"""GPU: the softmax of the shared-prefix decode where its reference moves often or
is hard to place, against fp64 attention over the oracle's dequantized tokens (setup
and error bounds of test_gpu_prefix_decode).

Many sequences read one and the same cache here: each CTA of the kernel then has
several tiles of a sequence, as with a long context, while the oracle has few tokens
to work out.
"""
import numpy as np
import pytest
import torch

import synth
from test_gpu_prefix_decode import DEV, Setup, check, contiguous, reference

pytestmark = pytest.mark.gpu


def one_cache(S, n, batch, data):
    """A layer of `batch` sequences that all read the same n tokens."""
    L = contiguous(S, [n], [data])
    Q = contiguous(S, [0] * batch, [([], [])] * batch, extra=8)
    Q.cache_ptrs.copy_(L.cache_ptrs.expand(batch))
    Q.lens.fill_(n)
    Q.cap = L.cap
    Q.keep = L  # the caches
    return Q


def ascending(S, n, step):
    """Tokens and a query direction (unit, [128]) whose base-2 logits rise by `step`
    per record of 32 tokens, from -step n / 64 to step n / 64."""
    sig = np.sqrt(np.concatenate([S.E[0], S.E[0]]) / 2)
    u = S.rng.standard_normal(128) * sig
    u /= np.linalg.norm(u)
    c = step * np.log(2.0) * (np.arange(n) // 32 - n / 64 + 0.5)
    k = c[:, None] * (u + 0.1 * S.rng.standard_normal((n, 128)) * sig / np.linalg.norm(sig))
    v = S.rng.standard_normal((n, 128))
    return (synth.to_bf16_bits(k[:, None]), synth.to_bf16_bits(v[:, None])), u


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shared", [False, True])
def test_reference_moves_in_every_chunk(shared, dtype):
    """Every 32-token chunk of every tile passes the one before by 2^9, so that each
    moves the reference: O of the tiles before and the tile's earlier weights are
    rescaled up to four times a tile. shared: a prefix behind more than 128 query rows
    of a KV head; else each sequence's own tokens."""
    S = Setup(41, 1, 4, 3)
    n, G = 1407, 16 if shared else 4
    B = 2048 if shared else 128  # about 10 tiles to a CTA
    data, u = ascending(S, n, 9.0)
    q = np.sqrt(128) * u + 0.1 * S.rng.standard_normal((B, G, 128))
    q = torch.from_numpy(q).to(dtype)
    if shared:
        P, Q = contiguous(S, [n], [data]), contiguous(S, [0] * B, [([], [])] * B, extra=8)
    else:
        P, Q = contiguous(S, [0], [([], [])]), one_cache(S, n, B, data)
    gs = torch.tensor([0, B], dtype=torch.int32, device=DEV)
    got = Q.decode_prefix(q.to(DEV), P, gs)
    assert Q.flags() == 0
    some = sorted(set(range(0, B, max(1, B // 40))) | {B - 1})
    heads, none = S.heads(*data), S.heads([], [])
    ref, tol = reference(S, q[some].double().numpy(), [none], [heads] * len(some),
                         [0] * len(some), dtype)
    check(got[some], ref, tol)
    assert torch.equal(Q.decode_prefix(q.to(DEV), P, gs), got)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [128, 600])
@pytest.mark.parametrize("sinks,norm,lead", [(1, 0.0, 12.0), (1, 0.0, 20.0), (1, 0.01, 20.0),
                                             (1, 0.0, 35.0), (32, 0.0, 20.0), (40, 0.01, 16.0)])
def test_heavy_tokens_of_small_value_norm(sinks, norm, lead, n, dtype):
    """Attention sinks: the first keys lead every logit by `lead` nats and their values
    are zero or far smaller than the others', which then carry the output.

    Bound on the error's norm, with B = sum_t p_t |v_hat_t|: logits off by d = 2^-19 D
    (bf16: 2^-11 D) and weights by e (as in test_gpu_prefix_decode) move the output by at
    most (exp(2 d) - 1 + e) B; a weight times norm below fp16's normal range is off by
    2^-25 at most where the largest is 2^5 or more, by 2^-30 of it each, at most 2^-29 n B
    in all (a token's centroids have between 0.5 and 2 times the norm sqrt(128)); storing
    adds half a step of the output's norm."""
    S = Setup(43, 1, 4, 4)
    sig = np.sqrt(np.concatenate([S.E[0], S.E[0]]) / 2)
    sig /= np.linalg.norm(sig)
    u = S.rng.standard_normal(128) * sig
    u /= np.linalg.norm(u)
    k, v = 3.0 * S.rng.standard_normal((n, 128)) * sig, S.rng.standard_normal((n, 128))
    k[:sinks] = lead * (u + 0.01 * S.rng.standard_normal((sinks, 128)) * sig)
    v[:sinks] *= norm
    data = synth.to_bf16_bits(k[:, None]), synth.to_bf16_bits(v[:, None])
    q = np.sqrt(128) * u + 0.1 * S.rng.standard_normal((2, 5, 128))
    q = torch.from_numpy(q).to(dtype)
    gs = torch.tensor([0, 2], dtype=torch.int32, device=DEV)
    none = ([], [])
    Q = one_cache(S, n, 2, data)
    got = Q.decode_prefix(q.to(DEV), contiguous(S, [0], [none]), gs)
    # the same tokens as the shared part
    pre = contiguous(S, [0, 0], [none, none], extra=8).decode_prefix(
        q.to(DEV), contiguous(S, [n], [data]), gs)
    assert torch.equal(pre, got) and Q.flags() == 0
    kh, vh = S.heads(*data)[0]
    got, q = got.double().cpu().numpy(), q.double().numpy()
    for b in range(2):
        for g in range(5):
            s = kh @ q[b, g] / np.sqrt(128)
            p = np.exp(s - s.max())
            p /= p.sum()
            ref, B = p @ vh, p @ np.linalg.norm(vh, axis=1)
            D = (np.abs(kh) @ np.abs(q[b, g])).max() / np.sqrt(128)
            bf16 = dtype == torch.bfloat16
            d, e = (2.0 ** -11 * D, 2.0 ** -11) if bf16 else (2.0 ** -19 * D,
                                                             2.0 ** -22 + n * 2.0 ** -26)
            u_out = 2.0 ** -8 if bf16 else 2.0 ** -24
            tol = (np.expm1(2 * d) + e + n * 2.0 ** -29) * B + u_out * np.linalg.norm(ref)
            err = np.linalg.norm(got[b, g] - ref)
            assert err <= tol, (err / tol, err / np.linalg.norm(ref))
