"""Whole decode steps of a stack whose layers keep their caches in 4 bits and in bf16, with the block
mass, evictions between steps, eager and from a CUDA graph."""
import numpy as np
import pytest
import torch

import synth
from oracle import sparda_oracle as O
from tests import kv4_reference as R
from tests.parity import check_selection, to64

pytestmark = pytest.mark.gpu
G, H, D = 2, 16, 128


@pytest.fixture(scope="module")
def sb(cuda_ok):
    from block_sparse_attention_forecast_gb300 import build
    build.build()
    import block_sparse_attention_forecast_gb300.binding as b
    b.sparda_device_error(clear=True)
    return b


def _stack(sb, kv4, T_list, topk, max_ctx, seed, **kw):
    """A stack holding T-1 tokens per sequence, seq_len at the next token; the same inputs for the same seed."""
    from block_sparse_attention_forecast_gb300.step import DecodeStack
    n, B, hidden = len(kv4), len(T_list), 256
    shape = sb.Shape(n_groups=G, topk=topk, max_ctx=max_ctx, max_batch=B)
    layers = []
    cached = torch.tensor([t - 1 for t in T_list], dtype=torch.int32, device="cuda")
    for L in range(n):
        bf = sb.LayerKV.empty(shape)
        bf.k.copy_(synth.normal_bf16((B, G, max_ctx, D), seed, 1, L).cuda())
        bf.v.copy_(synth.normal_bf16((B, G, max_ctx, D), seed, 2, L).cuda())
        sb.sparda_compress_keys(shape, bf, cached, B)
        if kv4[L]:
            layer = sb.LayerKV4.empty(shape)
            layer.kv.fill_(0xff)
            sb.sparda_kv4_quantize(shape, layer, bf.k, bf.v, cached, B)
            layer.ck = bf.ck
            layers.append(layer)
        else:
            layers.append(bf)
    W = [synth.normal_bf16((G * D, hidden), seed, 3, L, std=0.02).cuda() for L in range(n)]
    st = DecodeStack(shape, layers, W[0], W[1:], B, **kw)
    st.seq_len.copy_(cached + 1)
    return st


def _inputs(st, seed, step):
    n, B = st.n_layers, st.batch
    st.h.copy_(synth.normal_bf16(tuple(st.h.shape), seed, 10, step).cuda())
    st.q.copy_(synth.normal_bf16((n, B, G * H, D), seed, 11, step).cuda())
    st.k_new.copy_(synth.normal_bf16((n, B, G, D), seed, 12, step).cuda())
    st.v_new.copy_(synth.normal_bf16((n, B, G, D), seed, 13, step).cuda())


def _held(sb, st, L, seq):
    """Layer L's keys and values as the attention reads them, float64."""
    layer = st.layers[L]
    if not st.kv4[L]:
        return to64(layer.k), to64(layer.v)
    k = torch.zeros((st.batch, G, st.shape.max_ctx, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    sb.sparda_kv4_dequantize(st.shape, layer, seq, st.batch, k, v)
    return to64(k), to64(v)


def _check_step(sb, st, seq, mass_before):
    """Selections against the stored compressed keys, outputs and masses against the held values."""
    torch.cuda.synchronize()
    assert sb.sparda_device_error(clear=True) == 0
    for L in range(st.n_layers):
        K, V = _held(sb, st, L, seq)
        for b in range(st.batch):
            T = int(seq[b])
            for g in range(G):
                sel = [int(x) for x in st.idx[L, b, g, :int(st.cnt[L, b, g])]]
                ck = to64(st.layers[L].ck[b, g, :O.num_windows(T - 1)])
                S = O.pool_to_blocks(ck @ to64(st.f[L, b, g]), (T - 1) // 64 + 1)
                check_selection(st.idx[L, b, g], int(st.cnt[L, b, g]), S, T, st.shape.topk)
                # a 4-bit layer's values are read back through bf16 here: 2^-8 more per value
                w = 2.0 ** -11 + 2.0 ** -8 if st.kv4[L] else 2.0 ** -8
                ref, tol, mass, mtol = R.attention(to64(st.q[L, b, H * g:H * g + H]), K[b, g], V[b, g], sel, T, w)
                assert (np.abs(to64(st.out[L, b, H * g:H * g + H]) - ref) <= tol).all(), (L, b, g)
                got = to64(st.mass[L, b, g])[sel] - mass_before[L, b, g][sel]
                assert (np.abs(got - mass) <= mtol * mass + 2.0 ** -22 * to64(st.mass[L, b, g])[sel]).all()


@pytest.mark.parametrize("graph", [False, True])
def test_steps_with_mass_and_eviction(sb, graph):
    T_list, topk, max_ctx, seed = [1500, 900], 8, 2048, 600
    st = _stack(sb, [True, False, True], T_list, topk, max_ctx, seed, block_mass=True, advance=True)
    assert st.mode == "streams" and st.mass.shape == (3, 2, G, 32)
    seq = st.seq_len.clone()
    if graph:
        state = [x.clone() for l in st.layers for x in ((l.kv, l.ck) if hasattr(l, "kv") else (l.k, l.v, l.ck))]
        st.capture()
        for x, y in zip((x for l in st.layers for x in ((l.kv, l.ck) if hasattr(l, "kv") else (l.k, l.v, l.ck))), state):
            x.copy_(y)
        st.seq_len.copy_(seq)
        st.mass.zero_()
    mass = to64(st.mass)
    for step in range(8):
        _inputs(st, seed, step)
        st.run()
        _check_step(sb, st, seq, mass)
        mass = to64(st.mass)
        seq = seq + 1
        assert torch.equal(st.seq_len, seq)
        if step == 3:
            # mean pooling of the stored keys before and after: kept blocks keep their values
            before = [_held(sb, st, L, seq - 1) for L in range(3)]
            kept = st.evict(10, recent=2)
            torch.cuda.synchronize()
            assert sb.sparda_device_error(clear=True) == 0
            n_old = [(int(t) - 2) // 64 + 1 for t in seq]
            want = torch.tensor([int(t) - 64 * max(0, n - 10) for t, n in zip(seq, n_old)], dtype=torch.int32)
            assert torch.equal(st.seq_len.cpu(), want)
            for L in range(3):
                K, V = _held(sb, st, L, st.seq_len - 1)
                for b in range(2):
                    for g in range(G):
                        blocks = R.kept_blocks(mass[L, b, g], n_old[b], 10, 2)
                        assert kept[L, b, g].tolist() == blocks
                        T = int(want[b]) - 1
                        rows = np.concatenate([np.arange(64 * j, 64 * j + 64) for j in blocks])[:T]
                        assert np.array_equal(K[b, g, :T], before[L][0][b, g, rows])
                        assert np.array_equal(V[b, g, :T], before[L][1][b, g, rows])
            seq = st.seq_len.clone()
            mass = to64(st.mass)


def test_graph_and_eager_steps_agree(sb):
    runs = []
    for graph in (False, True):
        st = _stack(sb, [True, True], [700, 130], 4, 1024, 610, advance=True)
        _inputs(st, 610, 0)
        if graph:
            kv = [l.kv.clone() for l in st.layers]
            ck = [l.ck.clone() for l in st.layers]
            st.capture()
            for l, x, y in zip(st.layers, kv, ck):
                l.kv.copy_(x)
                l.ck.copy_(y)
            st.seq_len.copy_(torch.tensor([700, 130], dtype=torch.int32))
        outs = []
        for step in range(3):
            _inputs(st, 610, step)
            st.run()
            torch.cuda.synchronize()
            outs.append((st.out.clone(), st.idx.clone()))
        runs.append(outs)
    for (o, i), (o2, i2) in zip(*runs):
        assert torch.equal(o, o2) and torch.equal(i, i2)


def test_stack_refuses(sb):
    with pytest.raises(ValueError):
        _stack(sb, [True, False], [100, 100], 4, 1024, 620).evict(4)
    from block_sparse_attention_forecast_gb300.step import DecodeStack
    shape = sb.Shape(n_groups=G, topk=4, max_ctx=1024, max_batch=1)
    layers = [sb.LayerKV.empty(shape), sb.LayerKV.empty(shape, on_host=True)]
    W = torch.zeros((G * D, 256), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        DecodeStack(shape, layers, W, [W], 1, block_mass=True)


@pytest.mark.parametrize("advance", [False, True])
def test_capture_adds_nothing_to_the_mass(sb, advance):
    """Captured and replayed once, a stack holds the mass of one eager step, on top of what it held before;
    the capture alone leaves the mass as it was."""
    T_list, seed = [700, 130], 630
    st = _stack(sb, [True, False], T_list, 4, 1024, seed, block_mass=True, advance=advance)
    _inputs(st, seed, 0)
    start = torch.rand(st.mass.shape, generator=torch.Generator().manual_seed(seed)).cuda()
    st.mass.copy_(start)
    st.run()                                                      # eager
    torch.cuda.synchronize()
    want = st.mass.clone()
    assert not torch.equal(want, start)
    again = _stack(sb, [True, False], T_list, 4, 1024, seed, block_mass=True, advance=advance)
    _inputs(again, seed, 0)
    again.mass.copy_(start)
    again.capture()
    torch.cuda.synchronize()
    assert torch.equal(again.mass, start)
    again.seq_len.copy_(torch.tensor(T_list, dtype=torch.int32))  # the same token once more
    again.run()
    torch.cuda.synchronize()
    assert sb.sparda_device_error(clear=True) == 0
    assert torch.equal(again.mass, want) and torch.equal(again.out, st.out)
