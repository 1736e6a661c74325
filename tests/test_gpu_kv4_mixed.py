"""Decode stacks that hold 4-bit layers beside offloaded ones, and 4-bit stacks with host I/O: the same
results, bit for bit, as the resident stack with its inputs on the device."""
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu
G, D = 2, 128


@pytest.fixture(scope="module")
def sb(cuda_ok):
    from block_sparse_attention_forecast_gb300 import build
    build.build()
    import block_sparse_attention_forecast_gb300.binding as b
    b.sparda_device_error(clear=True)
    return b


def _stack(sb, kinds, T_list, seed, **kw):
    """kinds: one letter per layer, "4" in 4 bits, "b" bf16, "o" bf16 in host memory. T-1 tokens are cached."""
    from block_sparse_attention_forecast_gb300.step import DecodeStack
    B, ctx, hidden = len(T_list), 2048, 256
    shape = sb.Shape(n_groups=G, topk=6, max_ctx=ctx, max_batch=B)
    cached = torch.tensor([t - 1 for t in T_list], dtype=torch.int32, device="cuda")
    layers = []
    for L, kind in enumerate(kinds):
        K, V = (synth.normal_bf16((B, G, ctx, D), seed, i, L) for i in (1, 2))
        layer = sb.LayerKV.empty(shape, on_host=kind == "o")
        layer.k.copy_(K)
        layer.v.copy_(V)
        if kind == "o":
            sb.fill_hot_from_host(layer, [t - 1 for t in T_list])
        sb.sparda_compress_keys(shape, layer, cached, B)
        if kind == "4":
            bf, layer = layer, sb.LayerKV4.empty(shape)
            layer.kv.fill_(0xff)
            sb.sparda_kv4_quantize(shape, layer, bf.k, bf.v, cached, B)
            layer.ck = bf.ck
        layers.append(layer)
    W = [synth.normal_bf16((G * D, hidden), seed, 3, L, std=0.02).cuda() for L in range(len(kinds))]
    st = DecodeStack(shape, layers, W[0], W[1:], B, **kw)
    st.seq_len.copy_(cached + 1)
    return st


def _inputs(dst, seed, step):
    for i, name in enumerate(("h", "q", "k_new", "v_new")):
        dst[name].copy_(synth.normal_bf16(tuple(dst[name].shape), seed, 10 + i, step))


NAMES = ("h", "q", "k_new", "v_new")


@pytest.mark.parametrize("block_cache", [None, 16])
@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("kinds", ["4o4bo4", "bo44o", "4ooo4"])
def test_offloaded_layers_beside_4_bit_ones(sb, kinds, graph, block_cache):
    T_list, seed, steps = [1500, 126, 700], 640, 5     # (a block and a window fill on the way)
    runs = []
    for host in (False, True):
        st = _stack(sb, kinds if host else kinds.replace("o", "b"), T_list, seed, advance=True,
                    block_cache=block_cache if host else None)
        assert st.mode == "streams"
        if graph and host:
            # the warm-up step is the first one
            _inputs({n: getattr(st, n) for n in NAMES}, seed, 0)
            st.capture()
        out = []
        for step in range(1 if graph and host else 0, steps):
            _inputs({n: getattr(st, n) for n in NAMES}, seed, step)
            st.run()
            torch.cuda.synchronize()
            out.append((st.out.clone(), st.idx.clone(), st.seq_len.clone()))
        assert sb.sparda_device_error(clear=True) == 0
        runs.append((out, [l.ck.clone() for l in st.layers]))
    for a, b in zip(reversed(runs[0][0]), reversed(runs[1][0])):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert all(torch.equal(x, y) for x, y in zip(runs[0][1], runs[1][1]))


@pytest.mark.parametrize("kinds,mass", [("444444", False), ("444444", True), ("4b4b44", False), ("4b4b44", True),
                                        ("4o44o4", False)])
def test_host_io_of_4_bit_stacks(sb, kinds, mass):
    """Six layers: some inputs come by the copy kernel, some by DMA, and outputs leave by both."""
    T_list, seed, steps = [1500, 126, 700], 650, 4
    kw = dict(advance=True, block_mass=mass)
    plain, host, captured = (_stack(sb, kinds, T_list, seed, **kw) for _ in range(3))
    io = {}
    for st in (host, captured):
        io[st] = (st.pinned_inputs(), torch.zeros_like(st.out, device="cpu").pin_memory())
        st.attach_host_io(*io[st])
    for step in range(steps):
        _inputs({n: getattr(plain, n) for n in NAMES}, seed, step)
        plain.run()
        for st in (host, captured):
            _inputs(io[st][0], seed, step)
        host.run()
        if step == 0:
            captured.capture()                     # its warm-up step is the first one
        else:
            captured.run()
        torch.cuda.synchronize()
        for st in (host, captured):
            assert torch.equal(io[st][1], plain.out.cpu()) and torch.equal(st.idx, plain.idx), step
            assert torch.equal(st.seq_len, plain.seq_len)
    assert sb.sparda_device_error(clear=True) == 0
    if mass:
        assert torch.equal(host.mass, plain.mass)
