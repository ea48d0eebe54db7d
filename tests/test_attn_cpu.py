"""The attention layers' boundary without a GPU: the header is C99, the library exports what it
declares, sizes follow the format, bad arguments are refused before any device work; and the
oracle's 4-bit format against its description."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

from oracle import attn_oracle as ao

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fmoe_attn.h")


@pytest.fixture(scope="module")
def attn():
    from bit_dequant_expert_softmax_b200 import attn, build
    build.build()
    return attn


def test_header_is_plain_c99():
    out = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-x", "c", HEADER], capture_output=True,
                         text=True)
    assert out.returncode == 0, out.stderr


def test_exports_every_declared_symbol(attn):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(fmoe_[a-z_]+)\s*\(", src)))
    assert names == sorted(attn.EXPORTS)
    for n in names:
        assert hasattr(attn.lib(), n), n


@pytest.mark.parametrize("kv,D,P", [(8, 128, 64), (1, 64, 16), (3, 128, 1024)])
def test_page_bytes(attn, kv, D, P):
    cfg = attn.fmoe_attn_config(kv * 4, kv, D, P)
    # half a byte per channel of key and value, 4 bytes per group of 64
    assert attn.fmoe_kv_page_bytes(cfg) == kv * P * 2 * (D // 2 + D // 64 * 4) == ao.cache_bytes(kv, D, P)
    assert attn.fmoe_attn_workspace_bytes(cfg) > 0


@pytest.mark.parametrize("fields,status", [
    ((4, 0, 128, 64), 1), ((0, 1, 128, 64), 1), ((5, 2, 128, 64), 1), ((129, 1, 128, 64), 1), ((4, 2, 128, 24), 1),
    ((4, 2, 128, 0), 1), ((4, 2, 128, 2048), 1), ((4, 2, 0, 64), 1), ((4, 2, 96, 64), 2), ((4, 2, 256, 64), 2)])
def test_bad_configs(attn, fields, status):
    cfg = attn.fmoe_attn_config(*fields)
    assert attn.fmoe_kv_page_bytes(cfg) == 0 and attn.fmoe_attn_workspace_bytes(cfg) == 0
    L, P = attn.lib(), 0x10000
    assert L.fmoe_kv_append(cfg.ref, P, 512, P, 512, P, 512, 1, None, 0, 0, None, P, P, 1, 2 * P, None, None, None) == status
    assert L.fmoe_kv_gather(cfg.ref, P, 1, P, 1, 1, None, P, 1, P, P, None, None) == status
    assert L.fmoe_attn_decode(cfg.ref, P, 512, P, 1, P, 1, P, 1, 1.0, P, P, 1 << 30, None, None) == status
    assert L.fmoe_attn_prompt(cfg.ref, P, 512, P, 512, P, 512, P, P, 1, 1, 1, 1.0, P, None, None) == status


def _call(fn, names, good, **change):
    """fn with the good arguments, some changed."""
    args = dict(zip(names, good))
    assert set(change) <= set(args)
    args.update(change)
    return fn(*[args[n] for n in names])


A, B = 0x10000, 0x4000000  # addresses that no refused call reads


def test_append_refusals(attn):
    cfg = attn.fmoe_attn_config(4, 2, 128, 64)
    names = "cfg q qs k ks v vs T rope known rotary pos slots cache pages qo ko err stream".split()
    good = [cfg.ref, A, 512, A, 256, A, 256, 3, A, 100, 64, A, A, B, 2, B, 2 * B, None, None]
    f = attn.lib().fmoe_kv_append
    assert _call(f, names, good, T=0) == 0
    for bad in (dict(cfg=None), dict(T=-1), dict(pages=-1), dict(rotary=24), dict(rotary=144), dict(rotary=-16),
                dict(q=None), dict(qo=None), dict(q=A + 8), dict(qs=504), dict(qs=516), dict(k=None), dict(ks=255),
                dict(v=A + 2), dict(vs=128), dict(slots=None), dict(slots=A + 4), dict(cache=None), dict(cache=B + 64),
                dict(rope=None), dict(rope=A + 8), dict(pos=None), dict(known=0), dict(qo=B + 8), dict(ko=B + 4),
                dict(err=A + 2),
                dict(qs=768, qo=A),        # in place with another stride
                dict(qo=A + 1024),         # one token further on in the input
                dict(ko=A + 16), dict(qo=B + 64, ko=B + 128), dict(v=B, vs=256)):
        assert _call(f, names, good, **bad) == 1, bad


def test_gather_refusals(attn):
    cfg = attn.fmoe_attn_config(4, 2, 128, 64)
    names = "cfg cache pages table width seqs first cu rows ko vo err stream".split()
    good = [cfg.ref, A, 2, A, 3, 2, None, A, 50, B, 2 * B, None, None]
    f = attn.lib().fmoe_kv_gather
    assert _call(f, names, good, seqs=0) == 0 and _call(f, names, good, rows=0) == 0
    for bad in (dict(cfg=None), dict(cache=None), dict(cache=A + 16), dict(pages=-1), dict(table=None), dict(width=0),
                dict(seqs=-1), dict(first=A + 1), dict(cu=None), dict(rows=-1), dict(rows=1 << 31), dict(ko=None),
                dict(vo=B + 8), dict(vo=B + 1024), dict(err=A + 1)):
        assert _call(f, names, good, **bad) == 1, bad


def test_decode_refusals(attn):
    cfg = attn.fmoe_attn_config(4, 2, 128, 64)
    size = attn.fmoe_attn_workspace_bytes(cfg)
    names = "cfg q qs cache pages table width lens seqs scale out ws bytes err stream".split()
    good = [cfg.ref, A, 512, A, 2, A, 3, A, 2, 0.1, B, B, size, None, None]
    f = attn.lib().fmoe_attn_decode
    assert _call(f, names, good, seqs=0) == 0
    assert _call(f, names, good, ws=None) == 4 and _call(f, names, good, bytes=size - 1) == 4
    for bad in (dict(cfg=None), dict(q=None), dict(q=A + 8), dict(qs=500), dict(cache=None), dict(pages=-1),
                dict(table=None), dict(width=0), dict(width=1 << 25), dict(lens=None), dict(seqs=-1),
                dict(scale=float("nan")), dict(out=None), dict(out=B + 8), dict(out=A + 1024), dict(ws=B + 128),
                dict(err=A + 2)):
        assert _call(f, names, good, **bad) == 1, bad


def test_prompt_refusals(attn):
    cfg = attn.fmoe_attn_config(4, 2, 64, 64)
    names = "cfg q qs k ks v vs cq ck seqs n m scale out err stream".split()
    good = [cfg.ref, A, 256, A, 128, A, 128, A, A, 2, 10, 10, 0.1, B, None, None]
    f = attn.lib().fmoe_attn_prompt
    assert _call(f, names, good, seqs=0) == 0 and _call(f, names, good, n=0) == 0
    for bad in (dict(cfg=None), dict(q=None), dict(q=A + 4), dict(qs=248), dict(k=None), dict(ks=132), dict(v=None),
                dict(vs=64), dict(cq=None), dict(ck=None), dict(seqs=-1), dict(n=-1), dict(m=-1), dict(n=1 << 31),
                dict(scale=float("nan")), dict(out=None), dict(out=B + 8), dict(out=A), dict(err=A + 3),
                dict(v=B + 4096, vs=128)):
        assert _call(f, names, good, **bad) == 1, bad


@pytest.mark.parametrize("scale", [2.0 ** 24, -2.0 ** 24, float("inf"), -float("inf")])
def test_scales_out_of_range(attn, scale):
    """Scores that would pass what fp32 holds."""
    cfg = attn.fmoe_attn_config(4, 2, 64, 64)
    size = attn.fmoe_attn_workspace_bytes(cfg)
    assert attn.lib().fmoe_attn_decode(cfg.ref, A, 256, A, 2, A, 3, A, 2, scale, B, B, size, None, None) == 1
    for k in (A, None):
        assert attn.lib().fmoe_attn_prompt(cfg.ref, A, 256, k, 128, k, 128, A, A, 2, 10, 0, scale, B, None, None) == 1


def test_binding_refuses_wrong_tensors(attn):
    """Tensors of a wrong type, shape or place are refused by the binding (status 1)."""
    import torch
    from bit_dequant_expert_softmax_b200 import fmoe
    cfg = attn.fmoe_attn_config(4, 2, 64, 16)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    kv = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 3], dtype=torch.int32)
    for bad in (q, q.float(), q[..., :32], q.transpose(0, 1)):  # not on the GPU, fp32, short, other order
        with pytest.raises(fmoe.FmoeError) as e:
            attn.fmoe_attn_prompt(cfg, bad, kv, kv, cu, cu, q, 0.1)
        assert e.value.status == 1


@pytest.mark.parametrize("D", [64, 128])
def test_oracle_format(D):
    """Rows stored and loaded: every code within half a step of its value, at its place."""
    rng = np.random.default_rng(D)
    P, KV = 32, 3
    cache = np.full((4, ao.cache_bytes(KV, D, P)), 0xEE, np.uint8)
    rows = ao.bf16_round(rng.standard_normal((20, 2, KV, D)).astype(np.float32))
    table = np.array([2, 0])
    for t in range(20):
        t_at = t + 14  # over a tile and a page boundary
        slot = table[t_at // P] * P + t_at % P
        for w in range(2):
            for h in range(KV):
                ao.store(cache, P, slot, h, w, rows[t, w, h])
    for w, (c, s, b) in enumerate(ao.load(cache, D, P, table, 34)):
        got = (c * s + b)[:, 14:].transpose(1, 0, 2)
        step = s[:, 14:].transpose(1, 0, 2)
        # half a step, and the scale's own rounding over 15 steps
        assert (np.abs(got - rows[:, w]) <= step * (0.5 + 15 * ao.U16)).all()
        assert c.min() >= 0 and c[:, 14:].max() == 15
    assert (cache[1] == 0xEE).all() and (cache[3] == 0xEE).all()


def test_oracle_attention_by_hand():
    """Two keys with weights 1/4 and 3/4; causal rows; a row that sees nothing."""
    k = np.zeros((2, 1, 64))
    k[1, 0, 0] = np.log(3.0)
    v = np.zeros((2, 1, 64))
    v[0, 0, 0], v[1, 0, 1] = 4.0, 4.0
    q = np.zeros((3, 1, 64))
    q[:, 0, 0] = 1.0
    o, _ = ao.prompt(q, k, v, 1.0)
    assert (o[0] == 0).all() and np.allclose(o[1, 0, :2], [4, 0]) and np.allclose(o[2, 0, :2], [1, 3])


def test_oracle_rotation_keeps_lengths_and_differences():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((1, 1, 64)).astype(np.float32)
    a = np.arange(50)[:, None] * 100.0 ** (-np.arange(0, 32, 2) / 32)
    table = np.stack([np.cos(a), np.sin(a)], 1).astype(np.float32)
    y = ao.rotate(np.repeat(x, 50, 0), table, np.arange(50))[:, 0].astype(np.float64)
    # a pair's length stays within three bf16 half-steps; channels beyond the rotary ones stay
    r = np.hypot(y[:, :16], y[:, 16:32]) / np.hypot(x[0, 0, :16], x[0, 0, 16:32])
    assert np.abs(r - 1).max() < 3 * ao.U16 and (y[:, 32:] == x[0, 0, 32:]).all()
    # products depend on the difference of positions alone
    d = np.array([[y[i + j] @ y[i] for i in range(10)] for j in range(10)])
    assert np.abs(d - d[:, :1]).max() < 6 * ao.U16 * (x.astype(np.float64) ** 2).sum()
