"""Eviction of cache blocks by accumulated attention weight, bf16 and 4-bit caches, in place and into
another cache, against a plain restatement (tests/kv4_reference.py). Moves are compared byte for
byte, compressed keys with the exact means of the moved keys."""
import numpy as np
import pytest
import torch

import synth
from oracle import sparda_oracle as O
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


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _mass(B, G, nb, kind, seed):
    rng = np.random.default_rng(seed)
    if kind == "ties":
        m = rng.integers(0, 3, size=(B, G, nb)).astype(np.float32)
    elif kind == "zero":
        m = np.zeros((B, G, nb), dtype=np.float32)
        m[:, :, ::3] = -0.0
    else:
        m = np.exp(1.5 * rng.standard_normal((B, G, nb))).astype(np.float32)
        m[rng.random((B, G, nb)) < 0.3] = 0
    if kind == "special":
        m.reshape(-1)[::7] = np.nan
        m.reshape(-1)[3::11] = np.inf
        m.reshape(-1)[4::13] = -1.0
    return torch.from_numpy(m)


def _case(sb, kv4, T_list, G, ctx, mass_kind, seed):
    """(shape, layer, K as stored, mass) with one sequence behind the batch."""
    B = len(T_list) + 1
    shape = sb.Shape(n_groups=G, max_ctx=ctx, max_batch=B)
    K, V = synth.normal_bf16((B, G, ctx, 128), seed, 1), synth.normal_bf16((B, G, ctx, 128), seed, 2)
    bf = sb.LayerKV.empty(shape)
    bf.k.copy_(K.cuda())
    bf.v.copy_(V.cuda())
    full = _i32([min(max(t, 1), ctx) for t in T_list] + [ctx])
    sb.sparda_compress_keys(shape, bf, full, B)
    if not kv4:
        return shape, bf, K, _mass(B, G, ctx // 64, mass_kind, seed)
    layer = sb.LayerKV4.empty(shape)
    layer.kv.fill_(0x5a)
    sb.sparda_kv4_quantize(shape, layer, bf.k, bf.v, full, B)
    layer.ck.copy_(bf.ck)
    return shape, layer, torch.from_numpy(R.grid_values(K, True)), _mass(B, G, ctx // 64, mass_kind, seed)


def _planes(layer):
    """The cache's planes as byte tensors [B, G, nb, bytes per block]."""
    if hasattr(layer, "kv"):
        return [layer.kv]
    return [x.view(torch.uint8).view(*x.shape[:2], -1, 64 * 256) for x in (layer.k, layer.v)]


def _check(shape, before, after, K, mass, m_after, T_list, lens, kept, keep, recent, ck_before, dst_nb, untouched_ck):
    G = shape.n_groups
    for b, T in enumerate(T_list):
        n = (T - 1) // 64 + 1
        count = min(n, keep)
        assert int(lens[b]) == T - 64 * (n - count)
        W = O.num_windows(int(lens[b]))
        for g in range(G):
            m = mass[b, g].numpy()
            blocks = R.kept_blocks(m.astype(np.float64), n, keep, recent)
            assert [int(x) for x in kept[b, g]] == blocks + [-1] * (keep - count), (b, g)
            for x, y in zip(before, after):
                assert torch.equal(y[b, g, :count], x[b, g, blocks])
            got = m_after[b, g].numpy()
            assert np.array_equal(got[:count], m[blocks], equal_nan=True) and (got[count:dst_nb] == 0).all()
            want = untouched_ck[b, g].clone()
            for i, j in enumerate(blocks):
                for w in range(4):
                    if 4 * i + w >= W:
                        continue
                    if w < 3 or blocks[i + 1] == j + 1:
                        want[4 * i + w] = ck_before[b, g, 4 * j + w]
                    else:
                        span = np.concatenate([to64(K[b, g, 64 * j + 48:64 * j + 64]),
                                               to64(K[b, g, 64 * blocks[i + 1]:64 * blocks[i + 1] + 16])])
                        want[4 * i + w] = torch.from_numpy(O.compress_keys(span, 1)[0]).to(torch.bfloat16)
            yield b, g, want


CASES = [
    # T_list, G, ctx, keep, recent, weights
    ([1000, 64, 1, 640, 65], 2, 1024, 4, 1, "plain"),
    ([4096, 4095, 4033, 4032, 3000], 3, 4096, 17, 5, "plain"),
    ([4096, 2000], 1, 4096, 33, 32, "plain"),
    ([4000, 4096], 2, 4096, 40, 1, "ties"),
    ([4096], 2, 4096, 63, 2, "zero"),
    ([4096, 100], 2, 4096, 64, 2, "plain"),
    ([8000, 8192, 5000], 2, 8192, 21, 3, "special"),
    ([16384], 1, 16384, 200, 8, "plain"),
    ([2048] * 40, 4, 2048, 9, 2, "ties"),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_evict(sb, case, kv4, in_place):
    T_list, G, ctx, keep, recent, kind = CASES[case]
    B, nb = len(T_list), ctx // 64
    shape, layer, K, mass = _case(sb, kv4, T_list, G, ctx, kind, 200 + case)
    before = [x.cpu().clone() for x in _planes(layer)]
    ck_before = layer.ck.cpu().clone()
    m = mass.cuda()
    seq = _i32(T_list)
    kept = torch.full((B + 1, G, keep), -7, dtype=torch.int32, device="cuda")
    evict = sb.sparda_kv4_evict_blocks if kv4 else sb.sparda_evict_blocks
    if in_place:
        evict(shape, layer, m, seq, B, keep, recent, kept)
        after, m_after, lens, dst_nb, ck_after, untouched = layer, m, seq, nb, layer.ck, ck_before
    else:
        dshape = sb.Shape(n_groups=G, max_ctx=64 * (keep + 3), max_batch=B + 2)
        after = (sb.LayerKV4 if kv4 else sb.LayerKV).empty(dshape)
        for x in _planes(after):
            x.fill_(0x33)
        after.ck.fill_(5)
        untouched = after.ck.cpu().clone()
        dst_nb = keep + 3
        m_after = torch.full((B + 2, G, dst_nb), 11.0, device="cuda")
        lens = _i32([-1] * B)
        evict(shape, layer, m, seq, B, keep, recent, kept, dst_shape=dshape, dst=after, dst_mass=m_after, dst_seq_len=lens)
        ck_after = after.ck
    torch.cuda.synchronize()
    assert sb.sparda_device_error(clear=True) == 0
    planes = [x.cpu() for x in _planes(after)]
    got_ck = ck_after.cpu()
    seen = 0
    for b, g, want in _check(shape, before, planes, K, mass, m_after.cpu(), T_list, lens.cpu(), kept.cpu(), keep, recent,
                             ck_before, dst_nb, untouched):
        W = O.num_windows(int(lens[b]))
        assert torch.equal(got_ck[b, g, :W], want[:W]), (b, g)
        if not in_place:
            assert (got_ck[b, g, W:] == 5).all()
        seen += 1
    assert seen == B * G
    # the sequence behind the batch
    assert (kept[B] == -7).all()
    if in_place:
        for x, y in zip(before, planes):
            assert torch.equal(y[B], x[B])
        assert torch.equal(got_ck[B], ck_before[B])
        assert np.array_equal(m[B].cpu().numpy(), mass[B].numpy(), equal_nan=True)
    else:
        for x, y in zip(before, _planes(layer)):
            assert torch.equal(y.cpu(), x)                     # the source stays
        assert torch.equal(seq.cpu(), torch.tensor(T_list, dtype=torch.int32))
        assert (m_after[B:] == 11).all()
        for y in planes:
            assert (y[B:] == 0x33).all()


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_reports_bad_lengths(sb, in_place):
    shape, layer, _, mass = _case(sb, True, [1024, 1024, 1024], 2, 1024, "plain", 300)
    m, seq = mass.cuda(), _i32([0, 1024, 1025])
    kept = torch.zeros((3, 2, 4), dtype=torch.int32, device="cuda")
    before = layer.kv.clone()
    if in_place:
        sb.sparda_kv4_evict_blocks(shape, layer, m, seq, 3, 4, 1, kept)
        lens, after = seq, layer.kv
        same = before
    else:
        dshape = sb.Shape(n_groups=2, max_ctx=256, max_batch=3)
        dst = sb.LayerKV4.empty(dshape)
        dst.kv.fill_(0x33)
        same = dst.kv.clone()
        lens = _i32([9, 9, 9])
        sb.sparda_kv4_evict_blocks(shape, layer, m, seq, 3, 4, 1, kept, dst_shape=dshape, dst=dst,
                                   dst_mass=torch.zeros((3, 2, 4), device="cuda"), dst_seq_len=lens)
        after = dst.kv
    torch.cuda.synchronize()
    assert sb.sparda_device_error(clear=True) == sb.DEV_BAD_SEQ_LEN
    assert lens.tolist() == [0, 256, 1025]
    assert (kept[0] == -1).all() and (kept[2] == -1).all() and (kept[1] >= 0).all()
    assert torch.equal(after[0], same[0]) and torch.equal(after[2], same[2])


def test_evict_then_compress_agrees(sb):
    """After an in-place eviction of a bf16 cache the compressed keys are what sparda_compress_keys
    builds from the moved keys, and a second eviction continues from there (in a graph)."""
    T_list, G, ctx, keep = [4000, 3000], 2, 4096, 20
    shape, layer, _, mass = _case(sb, False, T_list, G, ctx, "plain", 400)
    m, seq = mass.cuda(), _i32(T_list)
    kept = torch.zeros((2, G, keep), dtype=torch.int32, device="cuda")
    sb.sparda_evict_blocks(shape, layer, m, seq, 2, keep, 4, kept)
    fresh = sb.LayerKV(layer.k, layer.v, torch.zeros_like(layer.ck))
    sb.sparda_compress_keys(shape, fresh, seq, 2)
    torch.cuda.synchronize()
    for b in range(2):
        W = O.num_windows(int(seq[b]))
        assert torch.equal(layer.ck[b, :, :W], fresh.ck[b, :, :W])
    graph = torch.cuda.CUDAGraph()
    k2 = torch.zeros((2, G, 9), dtype=torch.int32, device="cuda")
    with torch.cuda.graph(graph):
        sb.sparda_evict_blocks(shape, layer, m, seq, 2, 9, 2, k2)
    want = [R.kept_blocks(m[b, g, :].double().cpu().numpy(), (int(seq[b]) - 1) // 64 + 1, 9, 2) for b in range(2) for g in range(G)]
    kb = layer.k.clone()
    graph.replay()
    torch.cuda.synchronize()
    assert sb.sparda_device_error(clear=True) == 0
    for i, blocks in enumerate(want):
        b, g = divmod(i, G)
        assert k2[b, g].tolist() == blocks
        assert torch.equal(layer.k[b, g].view(-1, 64, 128)[:9], kb[b, g].view(-1, 64, 128)[blocks])
    graph.replay()                                             # nothing left to evict
    torch.cuda.synchronize()
    assert [int((t - 1) // 64 + 1) for t in seq.tolist()] == [9, 9] and k2[0, 0].tolist() == list(range(9))


def _bf16_mean(values):
    """The mean of 32 bf16 values (floats), exact, rounded once to bf16 (nearest even), as a float."""
    from fractions import Fraction
    s = sum((Fraction(float(v)) for v in values), Fraction(0)) / 32
    if s == 0:
        return 0.0
    a, e = abs(s), 0
    while a >= 2 ** (e + 1):
        e += 1
    while a < Fraction(2) ** e:
        e -= 1
    unit = Fraction(2) ** (max(e, -126) - 7)
    n = a / unit
    k = int(n)
    if n - k > Fraction(1, 2) or (n - k == Fraction(1, 2) and k & 1):
        k += 1
    return float(k * unit) * (1 if s > 0 else -1)


@pytest.mark.parametrize("spread", [0, 6, 20, 30, 60])
def test_joined_windows_are_exact_means(sb, spread):
    """Keys whose magnitudes spread over 2^+-spread, with zeros, cancellation and halfway sums: every
    joined window is the exact mean rounded once."""
    ctx, keep, seed = 1024, 5, 500 + spread
    shape = sb.Shape(n_groups=1, max_ctx=ctx, max_batch=1)
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((ctx, 128)) * 2.0 ** rng.integers(-spread, spread + 1, size=(ctx, 128))
    x[rng.random((ctx, 128)) < 0.05] = 0
    x[:, 1] = np.where(np.arange(ctx) % 2, 3.0, -3.0)                 # sums to nothing
    x[:, 2] = 0.0
    x[:, 3] = np.where(np.arange(ctx) % 32 == 5, 2.0 ** -3, 1.0 + 2.0 ** -7)  # sums near halfway
    x[:, 4] = 1.0
    x[:, 4][::16] = 1.0 + 2.0 ** -3                                   # 32 + 1/4: halfway in bf16 terms of the mean
    K = torch.from_numpy(x).to(torch.bfloat16)
    layer = sb.LayerKV.empty(shape)
    layer.k.copy_(K.cuda()[None, None])
    layer.v.zero_()
    mass = torch.zeros((1, 1, 16), device="cuda")
    mass[0, 0, [3, 6, 9]] = 1
    kept = torch.zeros((1, 1, keep), dtype=torch.int32, device="cuda")
    seq = _i32([ctx])
    sb.sparda_evict_blocks(shape, layer, mass, seq, 1, keep, 1, kept)
    torch.cuda.synchronize()
    blocks = [0, 3, 6, 9, 15]
    assert kept[0, 0].tolist() == blocks
    Kf = K.double().numpy()
    for i in range(keep - 1):
        span = np.concatenate([Kf[64 * blocks[i] + 48:64 * blocks[i] + 64], Kf[64 * blocks[i + 1]:64 * blocks[i + 1] + 16]])
        want = [_bf16_mean(span[:, c]) for c in range(128)]
        assert to64(layer.ck[0, 0, 4 * i + 3]).tolist() == want, i


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("lost", [1, 3, 200])
def test_evict_in_place_of_long_shifts(sb, kv4, lost):
    """Nearly every block moves by a few places, each onto one that moves too: the bytes of the old cache, the
    same in every run and in a replayed graph."""
    B, G, n = 2, 2, 1100
    keep, T = n - lost, 64 * n - 5
    shape = sb.Shape(n_groups=G, max_ctx=64 * n, max_batch=B)
    gen = torch.Generator(device="cuda").manual_seed(31)
    raw = torch.randint(0, 256, (B, G, n, 10240 if kv4 else 32768), generator=gen, dtype=torch.uint8, device="cuda")
    ck0 = torch.randint(-2 ** 14, 2 ** 14, (B, G, shape.w_cap, 128), generator=gen, dtype=torch.int16, device="cuda")

    def fresh():
        if kv4:
            return sb.LayerKV4(raw.clone(), ck0.clone().view(torch.bfloat16))
        k, v = (raw[..., i:i + 16384].contiguous().view(torch.bfloat16).view(B, G, 64 * n, 128) for i in (0, 16384))
        return sb.LayerKV(k, v, ck0.clone().view(torch.bfloat16))

    def held(layer):
        if kv4:
            return layer.kv
        return torch.cat([x.view(torch.uint8).view(B, G, n, 16384) for x in (layer.k, layer.v)], dim=-1)
    mass0 = torch.rand((B, G, n), generator=gen, device="cuda") + 1
    mass0[:, :, 1:1 + lost] = 0                            # the oldest go
    mass0[1, 1] = 1
    mass0[1, 1, torch.randperm(n - 2, generator=gen, device="cuda")[:lost] + 1] = 0
    want = []
    for b in range(B):
        for g in range(G):
            gone = set(torch.nonzero(mass0[b, g] == 0).flatten().tolist())
            want.append([j for j in range(n) if j not in gone])
    want = torch.tensor(want, device="cuda").view(B, G, keep)
    fn = sb.sparda_kv4_evict_blocks if kv4 else sb.sparda_evict_blocks
    kept = torch.empty((B, G, keep), dtype=torch.int32, device="cuda")
    layer, mass, seq = fresh(), mass0.clone(), torch.full((B,), T, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    for run in range(4):
        if run == 2:
            with torch.cuda.graph(graph):
                fn(shape, layer, mass, seq, B, keep, 1, kept)
        if run:
            again = fresh()
            for name in ("kv", "ck") if kv4 else ("k", "v", "ck"):
                getattr(layer, name).copy_(getattr(again, name))
            mass.copy_(mass0)
            seq.fill_(T)
        if run < 2:
            fn(shape, layer, mass, seq, B, keep, 1, kept)
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert sb.sparda_device_error(clear=True) == 0
        assert torch.equal(kept.long(), want)
        assert (seq == T - 64 * lost).all()
        got = held(layer)
        for b in range(B):
            for g in range(G):
                assert torch.equal(got[b, g, :keep], raw[b, g][want[b, g]]), (run, b, g)
                inner = torch.stack([ck0[b, g][4 * want[b, g] + i] for i in range(3)], dim=1)
                assert torch.equal(layer.ck[b, g].view(torch.int16)[:4 * keep - 1].view(-1, 128)[
                    (4 * torch.arange(keep, device="cuda")[:, None] + torch.arange(3, device="cuda")).flatten()].view(keep, 3, 128)
                    [:-1], inner[:-1]), (run, b, g)


def test_two_evictions_in_place_at_once(sb):
    """Two caches on two streams, each cut in place while the other is."""
    B, G, n, keep = 4, 2, 700, 450
    shape = sb.Shape(n_groups=G, max_ctx=64 * n, max_batch=B)
    gen = torch.Generator(device="cuda").manual_seed(41)
    streams = [torch.cuda.Stream() for _ in range(2)]
    raw = [torch.randint(0, 256, (B, G, n, 10240), generator=gen, dtype=torch.uint8, device="cuda") for _ in streams]
    mass0 = [torch.rand((B, G, n), generator=gen, device="cuda") + 1 for _ in streams]
    layers = [sb.LayerKV4(r.clone(), torch.zeros((B, G, shape.w_cap, 128), dtype=torch.bfloat16, device="cuda")) for r in raw]
    masses = [m.clone() for m in mass0]
    seqs = [torch.full((B,), 64 * n, dtype=torch.int32, device="cuda") for _ in streams]
    kept = [torch.empty((B, G, keep), dtype=torch.int32, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                layers[i].kv.copy_(raw[i])
                masses[i].copy_(mass0[i])
                seqs[i].fill_(64 * n)
                sb.sparda_kv4_evict_blocks(shape, layers[i], masses[i], seqs[i], B, keep, 3, kept[i])
    torch.cuda.synchronize()
    assert sb.sparda_device_error(clear=True) == 0
    for i in range(2):
        for b in range(B):
            for g in range(G):
                want = R.kept_blocks(mass0[i][b, g].cpu().numpy(), n, keep, 3)
                assert kept[i][b, g].tolist() == want
                assert torch.equal(layers[i].kv[b, g, :keep], raw[i][b, g][torch.tensor(want, device="cuda")])


@pytest.mark.parametrize("kv4", [False, True])
def test_evict_weights_of_the_batch_side_by_side(sb, kv4):
    """mass and dst_mass of fewer sequences than max_batch, neighbours in one tensor, either one first."""
    ctx, keep, G = 1024, 5, 2
    shape, layer, _, mass = _case(sb, kv4, [1000] * 5, G, ctx, "plain", 410)
    dshape = sb.Shape(n_groups=G, max_ctx=64 * keep, max_batch=5)
    fn = sb.sparda_kv4_evict_blocks if kv4 else sb.sparda_evict_blocks
    n_src, n_dst = 2 * G * 16, 2 * G * keep
    for first in (False, True):
        both = torch.full((n_src + n_dst + 8,), 3.0, device="cuda")
        m = both[n_dst:n_dst + n_src] if first else both[:n_src]
        dm = both[:n_dst] if first else both[n_src:n_src + n_dst]
        m.copy_(mass[:2].reshape(-1).cuda())
        kept = torch.zeros((2, G, keep), dtype=torch.int32, device="cuda")
        fn(shape, layer, m.view(2, G, 16), _i32([1000, 640]), 2, keep, 1, kept, dst_shape=dshape,
           dst=(sb.LayerKV4 if kv4 else sb.LayerKV).empty(dshape), dst_mass=dm.view(2, G, keep), dst_seq_len=_i32([0, 0]))
        torch.cuda.synchronize()
        assert sb.sparda_device_error(clear=True) == 0
        for b in range(2):
            for g in range(G):
                want = R.kept_blocks(mass[b, g].double().numpy(), (16, 10)[b], keep, 1)
                assert kept[b, g].tolist() == want
                assert torch.equal(dm.view(2, G, keep)[b, g].cpu(), mass[b, g][want])
        assert (both[-8:] == 3).all()


@pytest.mark.parametrize("kv4", [False, True])
def test_evict_in_place_whose_waits_run_out(sb, kv4, tmp_path, monkeypatch):
    """A build of the eviction that gives a wait up at its first look, over shifts by one block, in which nearly
    every write waits. The call reports it; a sequence of which a block was left keeps its length and
    weights, any other is cut as it should be."""
    from tests.test_launch_errors import compiled
    B, G, n = 5, 2, 700
    T = [64 * n - 3, 64 * n, 64 * (n - 1), 100, 64 * n - 60]          # two of them have nothing to move
    keep = n - 1
    lib = compiled(str(tmp_path), ["api.cu", "evict.cu", "attn.cu"], fake=None, extra=["-DSPARDA_SHIFT_POLLS=0"])
    shape = sb.Shape(n_groups=G, max_ctx=64 * n, max_batch=B)
    gen = torch.Generator(device="cuda").manual_seed(43)
    raw = torch.randint(0, 256, (B, G, n, 10240 if kv4 else 16384), generator=gen, dtype=torch.uint8, device="cuda")
    ck = torch.zeros((B, G, shape.w_cap, 128), dtype=torch.bfloat16, device="cuda")
    if kv4:
        layer = sb.LayerKV4(raw.clone(), ck)
    else:
        k = raw.clone().view(torch.bfloat16).view(B, G, 64 * n, 128)
        layer = sb.LayerKV(k, k.clone(), ck)
    mass0 = torch.rand((B, G, n), generator=gen, device="cuda") + 1
    mass0[:, :, 1] = 0                                                # the block to go, where one does
    mass, seq = mass0.clone(), _i32(T)
    kept = torch.full((B, G, keep), -7, dtype=torch.int32, device="cuda")
    monkeypatch.setattr(sb, "lib", lib)
    (sb.sparda_kv4_evict_blocks if kv4 else sb.sparda_evict_blocks)(shape, layer, mass, seq, B, keep, 1, kept)
    torch.cuda.synchronize()
    assert sb.sparda_device_error(clear=True) == sb.DEV_WAIT_TIMEOUT
    left = 0
    for b in range(B):
        cut = T[b] > 64 * keep
        blocks = [0] + list(range(2, n)) if cut else list(range((T[b] - 1) // 64 + 1))
        want = torch.tensor(blocks, device="cuda")
        if cut and int(seq[b]) == T[b]:
            left += 1
            assert torch.equal(mass[b], mass0[b])
        else:
            assert int(seq[b]) == T[b] - (64 if cut else 0)
            for g in range(G):
                m = torch.zeros(n, device="cuda")
                m[:len(blocks)] = mass0[b, g][want]
                assert torch.equal(mass[b, g], m)
                got = layer.kv[b, g] if kv4 else layer.k[b, g].reshape(n, -1).view(torch.uint8)
                assert torch.equal(got[:len(blocks)], raw[b, g][want])
        for g in range(G):
            assert kept[b, g].tolist() == blocks + [-1] * (keep - len(blocks))
    assert left >= 1


def _wide_windows(n, seed):
    """[n, 32] bf16 values (as floats) whose mean is lost unless all of every value counts: large ones that
    cancel beside small ones, over all exponents, subnormals, sums at and beside a tie, the largest values."""
    rng = np.random.default_rng(seed)
    sig = lambda size: rng.integers(128, 256, size=size).astype(np.float64) * rng.choice([-1.0, 1.0], size=size)
    x = np.zeros((n, 32))
    for i in range(n):
        kind = i % 6
        if kind == 0:                                    # a small rest behind what cancels
            pairs = rng.integers(1, 16)
            big = sig(pairs) * 2.0 ** rng.integers(-133, 121, size=pairs)
            x[i, :2 * pairs] = np.concatenate([big, -big])
            x[i, 2 * pairs:] = sig(32 - 2 * pairs) * 2.0 ** rng.integers(-133, 121)
        elif kind == 1:                                  # any exponents at all
            x[i] = sig(32) * 2.0 ** rng.integers(-133, 121, size=32)
        elif kind == 2:                                  # subnormals and a little more
            x[i] = rng.integers(-255, 256, size=32) * 2.0 ** -133
        elif kind == 3:                                  # a tie of the mean, and a last bit beside it or not
            e = rng.integers(-100, 100)
            x[i, 0], x[i, 1] = rng.integers(128, 256) * 2.0 ** e, 2.0 ** (e - 1)
            x[i, 2] = rng.integers(-1, 2) * 2.0 ** max(e - rng.integers(2, 60), -133)
            x[i, 3:5] = (2.0 ** 120, -2.0 ** 120)
        elif kind == 4:                                  # the largest
            x[i] = 255 * 2.0 ** 120 * (1 if i % 12 < 6 else rng.choice([-1.0, 1.0], size=32))
        else:
            x[i, :3] = (2.0 ** 60, 1.0, -2.0 ** 60)
        x[i] = rng.permutation(x[i])
    y = torch.from_numpy(x).to(torch.bfloat16)
    assert np.array_equal(y.double().numpy(), x)         # bf16 values as they stand
    return y


def test_joined_windows_of_any_magnitudes(sb):
    """As above for windows beyond every range that has a shorter way; infinities and NaN as a sum has them."""
    ctx, keep, lost = 64 * 40, 20, 20
    shape = sb.Shape(n_groups=2, max_ctx=ctx, max_batch=1)
    blocks = list(range(0, 38, 2)) + [39]
    rows = _wide_windows(2 * (keep - 1) * 128, 511).view(2, keep - 1, 128, 32)
    rows[0, 0, :4, 7] = torch.tensor([float("inf"), float("-inf"), float("nan"), float("inf")]).to(torch.bfloat16)
    rows[0, 0, 3, 8] = float("-inf")
    K = torch.zeros((1, 2, ctx, 128), dtype=torch.bfloat16)
    for i in range(keep - 1):
        a, b = 64 * blocks[i] + 48, 64 * blocks[i + 1]
        K[0, :, a:a + 16] = rows[:, i, :, :16].transpose(1, 2)
        K[0, :, b:b + 16] = rows[:, i, :, 16:].transpose(1, 2)
    mass = torch.zeros((1, 2, 40), device="cuda")
    mass[:, :, blocks[1:-1]] = 1
    for in_place in (True, False):
        layer = sb.LayerKV.empty(shape)
        layer.k.copy_(K.cuda())
        layer.v.zero_()
        kept, seq, m = torch.zeros((1, 2, keep), dtype=torch.int32, device="cuda"), _i32([ctx]), mass.clone()
        if in_place:
            sb.sparda_evict_blocks(shape, layer, m, seq, 1, keep, 1, kept)
            ck = layer.ck
        else:
            dshape = sb.Shape(n_groups=2, max_ctx=64 * keep, max_batch=1)
            dst = sb.LayerKV.empty(dshape)
            sb.sparda_evict_blocks(shape, layer, m, seq, 1, keep, 1, kept, dst_shape=dshape, dst=dst,
                                   dst_mass=torch.zeros((1, 2, keep), device="cuda"), dst_seq_len=_i32([0]))
            ck = dst.ck
        torch.cuda.synchronize()
        assert sb.sparda_device_error(clear=True) == 0
        assert kept[0, 0].tolist() == blocks and kept[0, 1].tolist() == blocks
        for g in range(2):
            for i in range(keep - 1):
                got, w = to64(ck[0, g, 4 * i + 3]), rows[g, i].double().numpy()
                for c in range(128):
                    with np.errstate(invalid="ignore"):
                        s = w[c].sum() if not np.isfinite(w[c]).all() else None
                    want = _bf16_mean(w[c]) if s is None else s
                    assert got[c] == want or (np.isnan(got[c]) and np.isnan(want)), (g, i, c, got[c], want)
                    # (a sum below zero whose mean rounds to nothing is -0, a sum of zero +0)
                    assert got[c] != 0 or np.signbit(got[c]) == np.signbit(want)


def test_append_of_windows_of_any_magnitudes(sb):
    """The compressed keys of the 4-bit append: groups of equal channels are stored as they stand, so that each
    window holds any 32 bf16 values."""
    B, G, n = 6, 4, 10                                    # windows per (sequence, group): every second one counted
    shape = sb.Shape(n_groups=G, max_ctx=64 * ((32 * n + 63) // 64), max_batch=B, heads_per_group=2)
    rows = _wide_windows(B * G * 4 * n, 521).view(B, G, 4, n, 32)
    tokens = rows.flatten(3).permute(3, 0, 1, 2)          # [32 n, B, G, 4]
    layer = sb.LayerKV4.empty(shape)
    zero = torch.zeros((B, G, 128), dtype=torch.bfloat16, device="cuda")
    keys = tokens.repeat_interleave(32, dim=3).contiguous().cuda()
    for t in range(32 * n):
        sb.sparda_kv4_append(shape, layer, keys[t], zero, _i32([t + 1] * B), B)
    torch.cuda.synchronize()
    assert sb.sparda_device_error(clear=True) == 0
    k = torch.zeros((B, G, shape.max_ctx, 128), dtype=torch.bfloat16, device="cuda")
    sb.sparda_kv4_dequantize(shape, layer, _i32([32 * n] * B), B, k, torch.zeros_like(k))
    assert torch.equal(k[:, :, :32 * n], keys.permute(1, 2, 0, 3))
    for b in range(B):
        for g in range(G):
            for c in range(4):
                for i in range(n):
                    want = _bf16_mean(rows[b, g, c, i].double().numpy())
                    assert to64(layer.ck[b, g, 2 * i, 32 * c:32 * c + 32]).tolist() == [want] * 32, (b, g, c, i)


def _compressed(sb, kv4, B, G, n, seed):
    """(shape, make, check) of caches of n full blocks whose compressed keys are the means of the keys as they are
    stored: make() is a fresh one, check(layer, seq) compares every complete window of it with the
    means of the keys that it holds now."""
    shape = sb.Shape(n_groups=G, max_ctx=64 * n, max_batch=B)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    bf = sb.LayerKV.empty(shape)
    bf.k.copy_(torch.randn(bf.k.shape, generator=gen, device="cuda"))
    bf.v.copy_(torch.randn(bf.v.shape, generator=gen, device="cuda"))
    full = _i32([64 * n] * B)
    layer = bf
    if kv4:
        layer = sb.LayerKV4.empty(shape)
        sb.sparda_kv4_quantize(shape, layer, bf.k, bf.v, full, B)
        sb.sparda_kv4_dequantize(shape, layer, full, B, bf.k, bf.v)
    sb.sparda_compress_keys(shape, bf, full, B)
    if kv4:
        layer.ck.copy_(bf.ck)

    def make():
        if kv4:
            return sb.LayerKV4(layer.kv.clone(), layer.ck.clone())
        return sb.LayerKV(layer.k.clone(), layer.v.clone(), layer.ck.clone())

    def check(got, seq):
        now = got
        if kv4:
            now = sb.LayerKV.empty(shape)
            sb.sparda_kv4_dequantize(shape, got, seq, B, now.k, now.v)
        want = sb.LayerKV(now.k, now.v, torch.zeros_like(got.ck))
        sb.sparda_compress_keys(shape, want, seq, B)
        torch.cuda.synchronize()
        for b in range(B):
            W = O.num_windows(int(seq[b]))
            assert torch.equal(got.ck[b, :, :W], want.ck[b, :, :W]), b
    return shape, make, check


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("lost", [1, 3, 200, 700])
def test_every_window_after_long_shifts(sb, kv4, lost):
    """The windows inside the moved blocks, those beside a neighbour that moved along and those formed anew, the
    last block's too, eager and replayed."""
    B, G, n = 2, 2, 1100
    keep = n - lost
    shape, make, check = _compressed(sb, kv4, B, G, n, 51)
    gen = torch.Generator(device="cuda").manual_seed(52)
    mass0 = torch.rand((B, G, n), generator=gen, device="cuda") + 1
    mass0[0, :, 1:1 + lost] = 0                            # one sequence loses its oldest blocks, one any
    fn = sb.sparda_kv4_evict_blocks if kv4 else sb.sparda_evict_blocks
    T = _i32([64 * n - 5, 64 * n])
    kept = torch.empty((B, G, keep), dtype=torch.int32, device="cuda")
    layer, mass, seq = make(), mass0.clone(), T.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fn(shape, layer, mass, seq, B, keep, 2, kept)
    for run in range(3):
        fresh = make()
        for name in ("kv", "ck") if kv4 else ("k", "v", "ck"):
            getattr(layer, name).copy_(getattr(fresh, name))
        mass.copy_(mass0)
        seq.copy_(T)
        if run:
            graph.replay()
        else:
            fn(shape, layer, mass, seq, B, keep, 2, kept)
        torch.cuda.synchronize()
        assert sb.sparda_device_error(clear=True) == 0
        assert seq.tolist() == [64 * keep - 5, 64 * keep]
        check(layer, seq)


def test_every_window_after_two_evictions_at_once(sb):
    """Two caches on two streams, one in 4 bits and one in bf16, each cut in place while the other is."""
    B, G, n, keep = 3, 2, 500, 320
    parts = []
    for kv4 in (False, True):
        shape, make, check = _compressed(sb, kv4, B, G, n, 53 + kv4)
        gen = torch.Generator(device="cuda").manual_seed(55 + kv4)
        mass = torch.rand((B, G, n), generator=gen, device="cuda")
        parts.append(dict(shape=shape, make=make, check=check, mass=mass, stream=torch.cuda.Stream(), runs=[],
                          fn=sb.sparda_kv4_evict_blocks if kv4 else sb.sparda_evict_blocks))
    for p in parts:
        p["runs"] = [dict(layer=p["make"](), mass=p["mass"].clone(), seq=_i32([64 * n, 64 * n - 40, 64 * n - 63]),
                          kept=torch.empty((B, G, keep), dtype=torch.int32, device="cuda")) for _ in range(4)]
    torch.cuda.synchronize()
    for i in range(4):
        for p in parts:
            with torch.cuda.stream(p["stream"]):
                r = p["runs"][i]
                p["fn"](p["shape"], r["layer"], r["mass"], r["seq"], B, keep, 3, r["kept"])
    torch.cuda.synchronize()
    assert sb.sparda_device_error(clear=True) == 0
    for p in parts:
        for r in p["runs"]:
            for b in range(B):
                for g in range(G):
                    assert r["kept"][b, g].tolist() == R.kept_blocks(p["mass"][b, g].cpu().numpy(), n, keep, 3)
            p["check"](r["layer"], r["seq"])
