"""The attention layers' entry points on the GPU (include/fmoe_attn.h) against the plain
definitions: the cache byte for byte, attention within the bound that the oracle derives from
the kernels' roundings."""
import numpy as np
import pytest
import torch

from oracle import attn_oracle as ao

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def attn(cuda_lib):
    from bit_dequant_expert_softmax_b200 import attn
    return attn


def _f32(t):
    return t.float().cpu().numpy()


def _f64(t):
    return t.double().cpu().numpy()


def _bf16(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16).cuda()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _filled(attn, cfg, pages, seed):
    """A cache of random codes, scales and biases."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    D, n = cfg.head_dim, cfg.head_dim // 64
    tb = 16 * (D + D // 8)
    cache = torch.randint(0, 256, (pages, attn.fmoe_kv_page_bytes(cfg)), generator=g, device="cuda", dtype=torch.uint8)
    sb = torch.empty(pages, cache.shape[1] // tb, 32 * n, 2, device="cuda")
    sb[..., 0] = torch.rand(sb.shape[:-1], generator=g, device="cuda") * 0.3 + 0.1
    sb[..., 1] = -torch.rand(sb.shape[:-1], generator=g, device="cuda") * 2 - 0.5
    cache.view(pages, -1, tb)[..., 16 * D:] = sb.to(torch.bfloat16).view(torch.uint8).flatten(2)
    return cache


def _table(rng, counts, P, pages, width=None):
    need = [-(-max(0, c) // P) for c in counts]
    order = rng.permutation(pages)[:sum(need)]
    t = np.full((len(counts), width or max(1, max(need))), -1, np.int32)
    at = 0
    for i, m in enumerate(need):
        t[i, :m] = order[at:at + m]
        at += m
    return t


def _close(got, ref, bound, what=""):
    bad = np.abs(got - ref) > bound + 1e-30
    assert np.isfinite(got).all() and not bad.any(), (
        f"{what}: {int((~np.isfinite(got)).sum())} not finite, worst error/bound "
        f"{np.nanmax(np.abs(got - ref) / np.maximum(bound, 1e-30)):.3f}")


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("H,KV,D,P,R,T,fused", [
    (4, 2, 128, 16, 128, 1, False), (32, 8, 128, 64, 64, 37, True), (6, 6, 64, 48, 64, 50, True),
    (14, 2, 64, 128, 32, 9, False), (5, 1, 128, 32, 0, 33, True), (3, 1, 64, 16, 16, 600, True)])
def test_append_bytes(attn, H, KV, D, P, R, T, fused):
    rng = np.random.default_rng(H * 1000 + T)
    cfg = attn.fmoe_attn_config(H, KV, D, P)
    x = _bf16(rng, T, H + 2 * KV, D)
    q, k, v = (y if fused else y.contiguous() for y in (x[:, :H], x[:, H:H + KV], x[:, H + KV:]))
    pages = -(-T // P) + 3
    cache = torch.full((pages, attn.fmoe_kv_page_bytes(cfg)), 0xA5, dtype=torch.uint8, device="cuda")
    slots = rng.permutation(pages * P)[:T]
    pos = rng.integers(0, 5000, T)
    rope = attn.rope_table(5000, R) if R else None
    qo = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
    ko = torch.empty(T, KV, D, dtype=torch.bfloat16, device="cuda")
    err = _err()
    attn.fmoe_kv_append(cfg, q, k, v, rope, _i32(pos), torch.from_numpy(slots).cuda(), cache, qo, ko, error=err)
    qr, kr = _f32(q), _f32(k)
    if R:
        table = rope.cpu().numpy()
        qr, kr = ao.rotate(qr, table, pos), ao.rotate(kr, table, pos)
    assert np.array_equal(_f32(qo), qr) and np.array_equal(_f32(ko), kr)
    want = np.full(cache.shape, 0xA5, np.uint8)
    vr = _f32(v)
    for t in range(T):
        for h in range(KV):
            ao.store(want, P, slots[t], h, 0, kr[t, h])
            ao.store(want, P, slots[t], h, 1, vr[t, h])
    assert np.array_equal(cache.cpu().numpy(), want)  # the other slots are as they were too
    assert int(err) == 0


@pytest.mark.parametrize("H,KV,D,P,R,T,fused", [(18, 2, 128, 64, 64, 1100, False), (18, 2, 128, 16, 128, 2400, True),
                                                (30, 1, 64, 32, 64, 1300, True)])
def test_append_many_tokens(attn, H, KV, D, P, R, T, fused):
    """So many that a token's heads lie in two blocks, or in one that goes round several times."""
    test_append_bytes(attn, H, KV, D, P, R, T, fused)


def test_append_in_place_without_queries_and_padding(attn):
    rng = np.random.default_rng(5)
    cfg = attn.fmoe_attn_config(4, 2, 128, 16)
    T, P = 7, 16
    q, k, v = _bf16(rng, T, 4, 128), _bf16(rng, T, 2, 128), _bf16(rng, T, 2, 128)
    rope = attn.rope_table(64, 128)
    pos = np.arange(T) + 3
    slots = np.array([3, -1, 40, 1 << 40, 17, 5, 6])
    pos[5] = 64  # outside the table
    err = _err()

    def fresh():
        return torch.zeros(3, attn.fmoe_kv_page_bytes(cfg), dtype=torch.uint8, device="cuda")

    q2, k2, a, b = q.clone(), k.clone(), fresh(), fresh()
    attn.fmoe_kv_append(cfg, q2, k2, v, rope, _i32(pos), torch.from_numpy(slots).cuda(), a, q2, k2, error=err)
    attn.fmoe_kv_append(cfg, None, k, v, rope, _i32(pos), torch.from_numpy(slots).cuda(), b)
    assert torch.equal(a, b)
    assert int(err) == attn.DEVERR_BAD_SLOT | attn.DEVERR_BAD_POSITION
    left = [1, 3, 5]
    rest = [0, 2, 4, 6]
    table = rope.cpu().numpy()
    for y, x in ((q2, q), (k2, k)):
        assert torch.equal(y[left], x[left])
        assert np.array_equal(_f32(y[rest]), ao.rotate(_f32(x[rest]), table, pos[rest]))
    want = np.zeros(a.shape, np.uint8)
    kr, vr = _f32(k2), _f32(v)
    for t in rest:
        for h in range(2):
            ao.store(want, P, slots[t], h, 0, kr[t, h])
            ao.store(want, P, slots[t], h, 1, vr[t, h])
    assert np.array_equal(a.cpu().numpy(), want)


def test_append_odd_values(attn):
    """Constant groups, the largest and smallest bf16 values, infinities and NaN."""
    cfg = attn.fmoe_attn_config(1, 1, 128, 16)
    big = float(torch.finfo(torch.bfloat16).max)
    rows = np.zeros((8, 128), np.float32)
    rows[1] = 3.5
    rows[2, ::2], rows[2, 1::2] = big, -big
    rows[3] = np.arange(128) * 2.0 ** -133
    rows[4, 5], rows[4, 70] = np.inf, 1.0
    rows[5, 64] = np.nan
    rows[6] = np.linspace(1.0, 1.0078125, 128)
    rows[7, 3] = -0.0
    v = torch.from_numpy(rows).to(torch.bfloat16).cuda().view(8, 1, 128)
    cache = torch.zeros(1, attn.fmoe_kv_page_bytes(cfg), dtype=torch.uint8, device="cuda")
    slots = torch.arange(8, device="cuda")
    attn.fmoe_kv_append(cfg, None, v, v, None, None, slots, cache)
    want = np.zeros(cache.shape, np.uint8)
    vr = _f32(v)[:, 0]
    for t in range(7):
        ao.store(want, 16, t, 0, 0, vr[t])
        ao.store(want, 16, t, 0, 1, vr[t])
    got = cache.cpu().numpy()
    kc, vc = torch.empty(8, 1, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(8, 1, 128, dtype=torch.bfloat16, device="cuda")
    attn.fmoe_kv_gather(cfg, cache, _i32([[0]]), _i32([0, 8]), kc, vc)
    back = _f32(kc)[:, 0]
    assert np.isnan(back[4, :64]).all() and np.isnan(back[5, 64:]).all()
    assert (back[[0, 7]] == 0).all() and (back[1] == 3.5).all() and np.isfinite(back[2]).all()
    assert torch.equal(kc.view(torch.int16), vc.view(torch.int16))
    sel = [i for i in range(8) if i != 7]  # row 7's bias is a zero of either sign
    for region, size in ((0, 64), (1024, 64), (2048, 8), (2176, 8)):
        for r in sel:
            at = region + r * size
            assert np.array_equal(got[0, at:at + size], want[0, at:at + size]), (region, r)


# ---------------------------------------------------------------- gather
@pytest.mark.parametrize("KV,D,P,counts,firsts", [
    (2, 128, 16, [1], [0]), (8, 64, 64, [0, 5, 0, 130, 1], [0, 3, 7, 60, 200]), (1, 128, 48, [100, 31], None),
    (3, 128, 1024, [7, 300], [1000, 0])])
def test_gather(attn, KV, D, P, counts, firsts):
    rng = np.random.default_rng(sum(counts))
    cfg = attn.fmoe_attn_config(KV, KV, D, P)
    f = firsts or [0] * len(counts)
    ends = [a + b for a, b in zip(f, counts)]
    pages = sum(-(-e // P) for e in ends) + 2
    cache = _filled(attn, cfg, pages, 3)
    table = _table(rng, ends, P, pages)
    cu = np.concatenate([[0], np.cumsum(counts)])
    n = int(cu[-1]) + 3  # three rows behind the last sequence
    ko, vo = (torch.full((n, KV, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    err = _err()
    attn.fmoe_kv_gather(cfg, cache, _i32(table), _i32(cu), ko, vo, first=None if firsts is None else _i32(f), error=err)
    assert int(err) == 0
    host = cache.cpu().numpy()
    for i, (a, c) in enumerate(zip(f, counts)):
        if c == 0:
            continue
        for out, (codes, s, b) in zip((ko, vo), ao.load(host, D, P, table[i], a + c)):
            ref = (codes * s + b)[:, a:].transpose(1, 0, 2)
            got = _f64(out[cu[i]:cu[i + 1]])
            # one fp32 rounding, then one to bf16
            assert (np.abs(got - ref) <= ao.U16 * np.abs(ref) * 1.001 + ao.U32 * (np.abs(codes * s) + np.abs(b))[:, a:].transpose(1, 0, 2)).all()
    assert (ko[cu[-1]:] == 7).all() and (vo[cu[-1]:] == 7).all()


def test_gather_leaves_bad_tokens_alone(attn):
    cfg = attn.fmoe_attn_config(2, 2, 64, 16)
    cache = _filled(attn, cfg, 3, 1)
    table = _i32([[0, 9], [2, 1]])
    ko, vo = (torch.full((60, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    err = _err()
    attn.fmoe_kv_gather(cfg, cache, table, _i32([0, 20, 60]), ko, vo, error=err)  # a bad page; 8 tokens too many
    assert int(err) == attn.DEVERR_BAD_PAGE | attn.DEVERR_BAD_LENGTH
    same = (ko == 7).all(-1).all(-1).cpu().numpy()
    assert same[16:20].all() and same[52:].all() and not same[:16].any() and not same[20:52].any()
    err.zero_()
    ko.fill_(7)
    attn.fmoe_kv_gather(cfg, cache, table, _i32([0, 10, 90]), ko, vo, first=_i32([0, -4]), error=err)
    assert int(err) == attn.DEVERR_BAD_LENGTH
    assert (ko[10:] == 7).all() and not (ko[:10] == 7).all()


# ---------------------------------------------------------------- decode
def _decode(attn, cfg, q, cache, table, lens, scale, workspace=None, error=None):
    out = torch.full((q.shape[0], cfg.q_heads, cfg.head_dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    attn.fmoe_attn_decode(cfg, q, cache, _i32(table), _i32(lens), out, scale,
                          attn.attn_workspace(cfg) if workspace is None else workspace, error=error)
    return out


def _check_decode(cfg, q, cache, table, lens, scale, out):
    host, qs, got = cache.cpu().numpy(), _f64(q), _f64(out)
    for s, n in enumerate(lens):
        ref, bound = ao.decode(qs[s], host, cfg.head_dim, cfg.page_tokens, table[s], n, scale)
        _close(got[s], ref, bound, f"sequence {s} of {n}")


@pytest.mark.parametrize("H,KV,D,P,lens", [
    (4, 1, 128, 16, [1]), (8, 8, 128, 64, [16, 0, 17]), (32, 8, 128, 64, [63, 64, 65, 1000]),
    (40, 8, 64, 16, [100, 1, 15, 0, 300]), (6, 2, 64, 48, [47, 48, 49]), (32, 2, 128, 128, [777]),
    (20, 1, 64, 32, [5, 130, 257]), (64, 1, 128, 16, [33, 2000]), (128, 1, 64, 1024, [1500]), (16, 2, 128, 64, [9000, 3])])
def test_decode(attn, H, KV, D, P, lens):
    rng = np.random.default_rng(H + sum(lens))
    cfg = attn.fmoe_attn_config(H, KV, D, P)
    pages = sum(-(-n // P) for n in lens) + 2
    cache, table = _filled(attn, cfg, pages, 11), _table(rng, lens, P, pages)
    q = _bf16(rng, len(lens), H, D)
    err = _err()
    out = _decode(attn, cfg, q, cache, table, lens, D ** -0.5, error=err)
    assert int(err) == 0
    _check_decode(cfg, q, cache, table, lens, D ** -0.5, out)


def test_decode_many_short_sequences(attn):
    """More (sequence, head) pairs than blocks, lengths zero to a few tiles, strided queries."""
    rng = np.random.default_rng(2)
    cfg = attn.fmoe_attn_config(16, 4, 128, 32)
    lens = [int(x) for x in rng.integers(0, 90, 333)]
    pages = sum(-(-n // 32) for n in lens)
    cache, table = _filled(attn, cfg, pages, 12), _table(rng, lens, 32, pages, width=9)
    q = _bf16(rng, 333, 24, 128)[:, :16]
    out = _decode(attn, cfg, q, cache, table, lens, 0.1)
    _check_decode(cfg, q, cache, table, lens, 0.1, out)


def test_decode_ignores_what_lies_behind_the_length(attn):
    """NaN in the slots behind a sequence, in other sequences' pages and in its own last tile."""
    rng = np.random.default_rng(3)
    cfg = attn.fmoe_attn_config(8, 2, 128, 32)
    lens = [33, 40, 7]
    cache = torch.full((9, attn.fmoe_kv_page_bytes(cfg)), 0xFF, dtype=torch.uint8, device="cuda")  # NaN words
    table = _table(rng, lens, 32, 9)
    slots = np.concatenate([table[s, np.arange(n) // 32].astype(np.int64) * 32 + np.arange(n) % 32 for s, n in enumerate(lens)])
    k, v = _bf16(rng, len(slots), 2, 128), _bf16(rng, len(slots), 2, 128)
    k[40, 1, 5] = float("inf")  # sequence 1, head 1
    attn.fmoe_kv_append(cfg, None, k, v, None, None, torch.from_numpy(slots).cuda(), cache)
    q = _bf16(rng, 3, 8, 128)
    out = _decode(attn, cfg, q, cache, table, lens, 0.09)
    host, qs, got = cache.cpu().numpy(), _f64(q), _f64(out)
    for s, n in enumerate(lens):
        for kv in range(2):
            heads = slice(4 * kv, 4 * kv + 4)
            if (s, kv) == (1, 1):
                assert np.isnan(got[s, heads]).all()
                continue
            one = host.reshape(9, 2, -1)[:, kv]
            ref, bound = ao.decode(qs[s, heads], one, 128, 32, table[s], n, 0.09)
            _close(got[s, heads], ref, bound, f"{s} {kv}")


def test_decode_bad_pages_and_lengths(attn):
    rng = np.random.default_rng(4)
    cfg = attn.fmoe_attn_config(4, 1, 64, 16)
    cache = _filled(attn, cfg, 4, 5)
    q = _bf16(rng, 4, 4, 64)
    table = np.array([[0, 1], [2, 4], [-3, 5], [3, 0]], np.int32)
    err = _err()
    out = _decode(attn, cfg, q, cache, table, [20, 30, 32, -5], 0.125, error=err)
    assert int(err) == attn.DEVERR_BAD_PAGE
    _check_decode(cfg, q[:1], cache, table, [20], 0.125, out[:1])
    _check_decode(cfg, q[1:2], cache, table[1:], [16], 0.125, out[1:2])  # the keys of its good page
    assert (out[2:] == 0).all()
    err.zero_()
    out = _decode(attn, cfg, q[:1], cache, table[3:], [500], 0.125, error=err)  # cut to the table's 32
    assert int(err) == attn.DEVERR_BAD_LENGTH
    _check_decode(cfg, q[:1], cache, table[3:], [32], 0.125, out)


def test_decode_large_scores(attn):
    """Scores far apart: one key takes all the weight; a scale of zero: all keys alike."""
    rng = np.random.default_rng(6)
    cfg = attn.fmoe_attn_config(8, 1, 128, 64)
    cache, table, lens = _filled(attn, cfg, 8, 8), np.arange(8, dtype=np.int32)[None], [500]
    q = _bf16(rng, 1, 8, 128, scale=100.0)
    for scale in (1.0, 0.0, -0.5):
        out = _decode(attn, cfg, q, cache, table, lens, scale)
        _check_decode(cfg, q, cache, table, lens, scale, out)


def test_decode_far_pages(attn):
    """Pages beyond 4 GiB of the cache."""
    rng = np.random.default_rng(7)
    cfg = attn.fmoe_attn_config(8, 8, 128, 128)
    pages = (5 << 30) // attn.fmoe_kv_page_bytes(cfg)
    big = torch.empty(pages, attn.fmoe_kv_page_bytes(cfg), dtype=torch.uint8, device="cuda")
    small = _filled(attn, cfg, 3, 9)
    big[-3:] = small
    q = _bf16(rng, 1, 8, 128)
    near, far = np.array([[2, 0, 1]], np.int32), np.array([[2, 0, 1]], np.int32) + pages - 3
    a = _decode(attn, cfg, q, small, near, [300], 0.1)
    b = _decode(attn, cfg, q, big, far, [300], 0.1)
    assert torch.equal(a, b)
    _check_decode(cfg, q, small, near, [300], 0.1, a)
    rows = [torch.empty(300, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    attn.fmoe_kv_gather(cfg, small, _i32(near), _i32([0, 300]), rows[0], rows[1])
    attn.fmoe_kv_gather(cfg, big, _i32(far), _i32([0, 300]), rows[2], rows[3])
    assert torch.equal(rows[0], rows[2]) and torch.equal(rows[1], rows[3])
    big[-3:] = 0
    slots = torch.from_numpy(far[0, np.arange(300) // 128].astype(np.int64) * 128 + np.arange(300) % 128).cuda()
    attn.fmoe_kv_append(cfg, None, rows[0], rows[1], None, None, slots, big)
    attn.fmoe_kv_gather(cfg, big, _i32(far), _i32([0, 300]), rows[2], rows[3])
    ref = [np.array([[(lambda c, s, b: (c * s[:, None] + b[:, None]).reshape(-1))(*ao.quantise(h.reshape(2, 64))) for h in r]
                     for r in _f32(x)]) for x in rows[:2]]
    for got, want in zip(rows[2:], ref):
        assert np.array_equal(_f32(got), ao.bf16_round(want))


def test_decode_two_streams_at_once(attn):
    """Calls on two streams at the same time, each with its own workspace."""
    rng = np.random.default_rng(14)
    cfg = attn.fmoe_attn_config(32, 8, 128, 64)
    cache = _filled(attn, cfg, 64, 4)
    jobs = []
    for i in range(2):
        lens = [900 + 100 * i, 0, 64, 333]
        table = _table(rng, lens, 64, 64)
        jobs.append((lens, table, _bf16(rng, 4, 32, 128), attn.attn_workspace(cfg), torch.cuda.Stream(), _i32(table), _i32(lens),
                     torch.empty(4, 32, 128, dtype=torch.bfloat16, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(20):
        for lens, _, q, ws, stream, t, n, out in jobs:
            attn.fmoe_attn_decode(cfg, q, cache, t, n, out, 0.1, ws, stream=stream)
    torch.cuda.synchronize()
    for lens, table, q, _, _, _, _, out in jobs:
        _check_decode(cfg, q, cache, table, lens, 0.1, out)


def test_decode_streams_and_graph(attn):
    """On another stream; captured once and replayed after the lengths and the cache changed;
    the same workspace with other sizes in between."""
    rng = np.random.default_rng(8)
    cfg = attn.fmoe_attn_config(16, 2, 128, 64)
    other = attn.fmoe_attn_config(64, 4, 64, 16)
    ws = attn.attn_workspace(cfg)
    assert attn.fmoe_attn_workspace_bytes(cfg) >= attn.fmoe_attn_workspace_bytes(other)
    cache, cache2 = _filled(attn, cfg, 40, 1), _filled(attn, other, 40, 2)
    lens = _i32([100, 1200])
    table_h = np.stack([np.arange(20), np.arange(20, 40)]).astype(np.int32)
    table = _i32(table_h)
    q = _bf16(rng, 2, 16, 128)
    out = torch.empty(2, 16, 128, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        attn.fmoe_attn_decode(cfg, q, cache, table, lens, out, 0.1, ws)
    torch.cuda.synchronize()
    _check_decode(cfg, q, cache, table_h, [100, 1200], 0.1, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        attn.fmoe_attn_decode(cfg, q, cache, table, lens, out, 0.1, ws)
    for now in ([100, 1200], [0, 1], [1280, 700]):
        lens.copy_(_i32(now))
        q.copy_(_bf16(rng, 2, 16, 128))
        graph.replay()
        torch.cuda.synchronize()
        _check_decode(cfg, q, cache, table_h, now, 0.1, out)
        q2 = _bf16(rng, 3, 64, 64)
        t2 = np.arange(30).reshape(3, 10).astype(np.int32)
        o2 = _decode(attn, other, q2, cache2, t2, [160, 3, 77], 0.1, workspace=ws)
        _check_decode(other, q2, cache2, t2, [160, 3, 77], 0.1, o2)
    a = out.clone()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, out)  # the same inputs give the same bits


# ---------------------------------------------------------------- prompt
def _check_prompt(q, k, v, cq, ck, scale, out):
    qs, ks, vs, got = _f64(q), _f64(k), _f64(v), _f64(out)
    for s in range(len(cq) - 1):
        a, b, c, d = cq[s], cq[s + 1], ck[s], ck[s + 1]
        ref, bound = ao.prompt(qs[a:b], ks[c:d], vs[c:d], scale)
        _close(got[a:b], ref, bound, f"sequence {s}: {b - a} queries, {d - c} keys")


@pytest.mark.parametrize("H,KV,D,lq,more", [
    (4, 2, 128, [1], [0]), (8, 8, 64, [127, 1, 0, 129], None), (32, 8, 128, [333], [0]),
    (40, 8, 64, [20, 300, 7], [100, 0, 513]), (6, 2, 128, [64, 65], [-30, 3]), (14, 2, 64, [50, 40], [-60, -40]),
    (128, 1, 64, [3, 40], [5, 0]), (33, 1, 128, [77], [200]), (24, 3, 128, [700, 513], [0, 1]), (1, 1, 64, [1500], [0]),
    # lengths around the steps of 64 and 128 keys
    (4, 1, 128, [63, 64, 65, 127, 128, 129, 191, 192, 193, 256, 257, 2], None),
    (7, 1, 64, [63, 64, 65, 127, 128, 129, 191, 192, 193], [1, 64, 0, 65, 128, 0, 63, 1, 2]),
    # long sequences and blocks for every SM: two row tiles per block
    (32, 8, 128, [1400], [0]), (40, 8, 64, [1300, 40], [300, -40]), (16, 16, 64, [2600], [-100]),
    (28, 4, 128, [1200, 900, 31], [0, 130, 2])])
def test_prompt(attn, H, KV, D, lq, more):
    rng = np.random.default_rng(H + sum(lq))
    cfg = attn.fmoe_attn_config(H, KV, D)
    lk = [max(0, a + b) for a, b in zip(lq, more or [0] * len(lq))]
    cq, ck = (np.concatenate([[0], np.cumsum(x)]) for x in (lq, lk))
    n, m = int(cq[-1]) + 2, int(ck[-1]) + 2  # rows behind the last sequence
    q, k, v = _bf16(rng, n, H, D, scale=2.0), _bf16(rng, m, KV, D), _bf16(rng, m, KV, D)
    k[-2:], v[-2:], q[-2:] = float("nan"), float("nan"), float("nan")
    out = torch.full((n, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    err = _err()
    attn.fmoe_attn_prompt(cfg, q, k, v, _i32(cq), _i32(ck), out, D ** -0.5, error=err)
    assert int(err) == 0 and (out[-2:] == 7).all()
    _check_prompt(q, k, v, cq, ck, D ** -0.5, out)


@pytest.mark.parametrize("H,KV,D,top,seqs", [(24, 8, 64, 260, 45), (16, 16, 128, 130, 40), (6, 6, 64, 600, 40), (40, 8, 128, 90, 70)])
def test_prompt_more_work_than_blocks_at_once(attn, H, KV, D, top, seqs):
    """Packed lengths of any kind, empty ones and queries without keys among them, several units to a block."""
    rng = np.random.default_rng(H + top)
    lq = [int(n) for n in rng.integers(0, top, seqs)]
    test_prompt(attn, H, KV, D, lq, [int(n) for n in rng.integers(-top, top // 2, seqs)])


def test_prompt_strides_and_other_sequences(attn):
    """Views of one fused buffer; NaN and infinities in the sequences around one."""
    rng = np.random.default_rng(9)
    cfg = attn.fmoe_attn_config(12, 4, 128)
    lens = [50, 131, 60, 200]
    cu = np.concatenate([[0], np.cumsum(lens)])
    x = _bf16(rng, int(cu[-1]), 20, 128)
    x[cu[0]:cu[1]] = float("nan")
    x[cu[2]:cu[3]] = float("inf")
    q, k, v = x[:, :12], x[:, 12:16], x[:, 16:]
    out = torch.empty(int(cu[-1]), 12, 128, dtype=torch.bfloat16, device="cuda")
    attn.fmoe_attn_prompt(cfg, q, k, v, _i32(cu), _i32(cu), out, 0.09)
    for s in (1, 3):
        a, b = cu[s], cu[s + 1]
        ref, bound = ao.prompt(_f64(q[a:b]), _f64(k[a:b]), _f64(v[a:b]), 0.09)
        _close(_f64(out[a:b]), ref, bound, f"sequence {s}")


def test_prompt_bad_offsets(attn):
    rng = np.random.default_rng(10)
    cfg = attn.fmoe_attn_config(4, 4, 64)
    q, k, v = (_bf16(rng, 100, 4, 64) for _ in range(3))
    out = torch.full((100, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    err = _err()
    # the second sequence runs past the rows, the third backwards
    attn.fmoe_attn_prompt(cfg, q, k, v, _i32([0, 30, 130, 90]), _i32([0, 30, 130, 90]), out, 0.1, error=err)
    assert int(err) == attn.DEVERR_BAD_LENGTH and (out[30:] == 7).all()
    _check_prompt(q, k, v, [0, 30], [0, 30], 0.1, out)


def test_prompt_without_any_key(attn):
    """Queries before the first key (no key rows at all): zeros, rows behind the last sequence left."""
    rng = np.random.default_rng(12)
    cfg = attn.fmoe_attn_config(6, 2, 128)
    q, none = _bf16(rng, 140, 6, 128), torch.empty(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    out = torch.full((140, 6, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    err = _err()
    attn.fmoe_attn_prompt(cfg, q, none, none, _i32([0, 130, 139]), _i32([0, 0, 0]), out, 0.1, error=err)
    assert int(err) == 0 and (out[:139] == 0).all() and (out[139] == 7).all()


def test_prompt_large_scores(attn):
    rng = np.random.default_rng(11)
    cfg = attn.fmoe_attn_config(2, 1, 128)
    q, k, v = _bf16(rng, 300, 2, 128, scale=60.0), _bf16(rng, 300, 1, 128), _bf16(rng, 300, 1, 128)
    for scale in (1.0, 0.0, -0.3):
        out = torch.empty(300, 2, 128, dtype=torch.bfloat16, device="cuda")
        attn.fmoe_attn_prompt(cfg, q, k, v, _i32([0, 300]), _i32([0, 300]), out, scale)
        _check_prompt(q, k, v, [0, 300], [0, 300], scale, out)


def test_prompt_two_streams_at_once(attn):
    """Two calls side by side, each with more blocks than fit: both as when alone."""
    rng = np.random.default_rng(21)
    cfg = attn.fmoe_attn_config(16, 8, 128)
    cu = _i32(np.concatenate([[0], np.cumsum(rng.integers(1, 200, 60))]))
    rows = int(cu[-1])
    jobs = [[_bf16(rng, rows, h, 128) for h in (16, 8, 8)] for _ in range(2)]
    alone = [attn.fmoe_attn_prompt(cfg, *j, cu, cu, torch.empty_like(j[0]), 0.09) for j in jobs]
    outs = [torch.empty_like(j[0]) for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(4):
        for j, out, stream in zip(jobs, outs, streams):
            attn.fmoe_attn_prompt(cfg, *j, cu, cu, out, 0.09, stream=stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(alone, outs))


def test_prompt_stream_graph_and_repeat(attn):
    rng = np.random.default_rng(12)
    cfg = attn.fmoe_attn_config(8, 2, 128)
    q, k, v = _bf16(rng, 400, 8, 128), _bf16(rng, 400, 2, 128), _bf16(rng, 400, 2, 128)
    cu = _i32([0, 150, 400])
    out = torch.empty(400, 8, 128, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        attn.fmoe_attn_prompt(cfg, q, k, v, cu, cu, out, 0.1)
    torch.cuda.synchronize()
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        attn.fmoe_attn_prompt(cfg, q, k, v, cu, cu, out, 0.1)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, out)
    cu.copy_(_i32([0, 399, 400]))
    graph.replay()
    torch.cuda.synchronize()
    _check_prompt(q, k, v, [0, 399, 400], [0, 399, 400], 0.1, out)


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("H,KV,D,P,R", [(8, 2, 128, 64, 64), (10, 5, 64, 16, 64)])
def test_a_layer_serving_two_sequences(attn, H, KV, D, P, R):
    """Prompts into the cache and through attention, one continued from its cached prefix, then
    single tokens over the cache: every output against the definition on what is cached."""
    rng = np.random.default_rng(13)
    cfg = attn.fmoe_attn_config(H, KV, D, P)
    rope, ws, scale = attn.rope_table(2048, R), attn.attn_workspace(cfg), D ** -0.5
    cache = attn.kv_cache(cfg, 64)
    table_h = _table(rng, [600, 300], P, 64, width=640 // P)
    table = _i32(table_h)
    have = [0, 0]

    def append(counts):
        """New tokens of each sequence -> rotated q and k, v, their places."""
        n = sum(counts)
        x = _bf16(rng, n, H + 2 * KV, D)
        at = np.concatenate([np.arange(h, h + c) for h, c in zip(have, counts)])
        seq = np.repeat([0, 1], counts)
        slots = table_h[seq, at // P].astype(np.int64) * P + at % P
        q, k = torch.empty(n, H, D, dtype=torch.bfloat16, device="cuda"), torch.empty(n, KV, D, dtype=torch.bfloat16, device="cuda")
        attn.fmoe_kv_append(cfg, x[:, :H], x[:, H:H + KV], x[:, H + KV:], rope, _i32(at), torch.from_numpy(slots).cuda(), cache, q, k)
        for i in range(2):
            have[i] += counts[i]
        return q, k, x[:, H + KV:]

    q, k, v = append([333, 150])
    cu = np.array([0, 333, 483])
    out = torch.empty_like(q)
    attn.fmoe_attn_prompt(cfg, q, k, v, _i32(cu), _i32(cu), out, scale)
    _check_prompt(q, k, v, cu, cu, scale, out)

    # sequence 0 goes on: its keys and values, old and new, come from the cache
    q, _, _ = append([100, 0])
    keys, vals = (torch.empty(have[0], KV, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    attn.fmoe_kv_gather(cfg, cache, table[:1], _i32([0, have[0]]), keys, vals)
    out = torch.empty_like(q)
    attn.fmoe_attn_prompt(cfg, q, keys, vals, _i32([0, 100]), _i32([0, have[0]]), out, scale)
    _check_prompt(q, keys, vals, [0, 100], [0, have[0]], scale, out)

    for _ in range(3):
        q, _, _ = append([1, 1])
        out = _decode(attn, cfg, q, cache, table_h, have, scale, workspace=ws)
        _check_decode(cfg, q, cache, table_h, have, scale, out)
