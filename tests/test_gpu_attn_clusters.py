"""The bf16 decode attention where a (sequence, group) is one thread-block cluster: clusters of 2 to 8
CTAs, many of them with nothing or almost nothing to attend, so that a CTA reaches the exchange of
partial results as early as it can."""
import numpy as np
import pytest
import torch

import synth
from tests import kv4_reference as R
from tests.parity import to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sb(cuda_ok):
    from block_sparse_attention_forecast_gb300 import build
    build.build()
    import block_sparse_attention_forecast_gb300.binding as b
    b.sparda_device_error(clear=True)
    return b


# (sequences, groups): 8, 8, 5, 4 and 2 CTAs per cluster on 152 SMs
@pytest.mark.parametrize("B,G", [(16, 1), (9, 2), (15, 2), (19, 2), (32, 2)])
@pytest.mark.parametrize("mass", [False, True])
def test_clusters_with_little_to_attend(sb, B, G, mass):
    topk, ctx, nb = 14, 1024, 16
    shape = sb.Shape(n_groups=G, max_ctx=ctx, max_batch=B, topk=topk)
    rng = np.random.default_rng(700 + B)
    K, V = synth.normal_bf16((B, G, ctx, 128), 701, 1), synth.normal_bf16((B, G, ctx, 128), 701, 2)
    layer = sb.LayerKV.empty(shape)
    layer.k.copy_(K.cuda())
    layer.v.copy_(V.cuda())
    q = synth.normal_bf16((B, 16 * G, 128), 702)
    T = rng.integers(1, ctx + 1, size=B)
    idx, cnt = np.full((B, G, topk + 2), -1, dtype=np.int32), np.zeros((B, G), dtype=np.int32)
    for b in range(B):
        n = (int(T[b]) - 1) // 64 + 1
        for g in range(G):
            # nothing, one block (all but one CTA of the cluster idle), or any number
            cnt[b, g] = (0, min(1, n), rng.integers(0, min(n, topk + 2) + 1))[(b * G + g) % 3]
            idx[b, g, :cnt[b, g]] = np.sort(rng.permutation(n)[:cnt[b, g]])
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    idx_d, cnt_d, seq, q_d = dev(idx), dev(cnt), dev(T.astype(np.int32)), q.cuda()
    ws = sb.workspace(shape, B, sb.WS_ATTN_MASS)
    runs = 20
    outs = [torch.full((B, 16 * G, 128), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(runs)]
    m = torch.zeros((runs, B, G, nb), device="cuda")
    for i in range(runs):                              # each may begin while the one before it ends
        if mass:
            sb.sparda_sparse_decode_attn_mass(shape, layer, q_d, idx_d, cnt_d, seq, B, outs[i], ws, m[i])
        else:
            sb.sparda_sparse_decode_attn(shape, layer, q_d, idx_d, cnt_d, seq, B, outs[i], ws)
    torch.cuda.synchronize()
    assert sb.sparda_device_error(clear=True) == 0
    for i in range(1, runs):
        assert torch.equal(outs[i], outs[0]) and torch.equal(m[i], m[0])
    got, got_m = to64(outs[0]), to64(m[0])
    for b in range(B):
        for g in range(G):
            blocks = [int(j) for j in idx[b, g, :cnt[b, g]]]
            ref, tol, w, wtol = R.attention(to64(q[b, 16 * g:16 * g + 16]), to64(K[b, g]), to64(V[b, g]), blocks,
                                            int(T[b]), 2.0 ** -8)
            assert (np.abs(got[b, 16 * g:16 * g + 16] - ref) <= tol).all(), (b, g)
            if mass:
                want = np.zeros(nb)
                want[blocks] = w
                assert (np.abs(got_m[b, g] - want) <= (wtol + 2.0 ** -22) * want).all(), (b, g)
