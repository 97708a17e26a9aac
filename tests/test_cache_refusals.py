"""The cache's operators refuse what they cannot do, with the documented status
and before any HIP call (no GPU is needed), and the binding with a ValueError."""
import array

import pytest
import torch

import reduction_codec_amd as rca

A, M = 0x10000, 0x10008                     # aligned, misaligned: never dereferenced


def cache(k=A, v=A, pages=4, page=16, kv=2, d=128, table=A, seqs=2, max_pages=4, lengths=A, offsets=A):
    return array.array("Q", [k or 0, v or 0, pages, page, kv, d, table or 0, seqs, max_pages, lengths or 0, offsets or 0])


def append(t=3, tokens=3, k=A, ks=256, v=A, vs=256, heads=4, q=A, qs=512, q_out=2 * A, rotation=A, positions=64, rot=128,
           null=False, **c):
    a = cache(**{n[2:]: x for n, x in c.items()})
    return rca.lib().rc_mxfp4_cache_append(None if null else a.buffer_info()[0], t, tokens, k, ks, v, vs, heads, q, qs,
                                           q_out, rotation, positions, rot, 0, None)


def read(t=3, tokens=3, k=A, v=A, null=False, **c):
    a = cache(**{n[2:]: x for n, x in c.items()})
    return rca.lib().rc_mxfp4_cache_read(None if null else a.buffer_info()[0], tokens, t, k, v, None)


def attend(t=3, tokens=3, heads=4, q=A, qs=512, causal=1, window=0, out=A, lse=A, ws=A, null=False, **c):
    a = cache(**{n[2:]: x for n, x in c.items()})
    return rca.lib().rc_mxfp4_cache_attention(None if null else a.buffer_info()[0], t, tokens, heads, q, qs, 0.1, causal,
                                              window, 0, out, lse, ws, None)


@pytest.mark.parametrize("call", [append, read, attend])
def test_cache(call):
    assert call(null=True) == rca.ERR_NULL and call(t=0) == rca.ERR_UNSUPPORTED and call(t=4) == rca.ERR_UNSUPPORTED
    for bad in ({"c_d": 0}, {"c_d": 32}, {"c_d": 80}, {"c_d": 160}, {"c_d": 512}, {"c_page": 8}, {"c_page": 48},
                {"c_page": 0}, {"c_page": 131072}, {"c_page": 32, "c_d": 96}, {"c_page": 16, "c_d": 64}, {"c_kv": 0},
                {"c_kv": 65536}, {"c_seqs": 65536}, {"c_pages": 1 << 31}, {"tokens": 1 << 31},
                {"c_max_pages": 1 << 27}, {"c_pages": 1 << 30, "c_kv": 1 << 10}, {"c_page": (1 << 64) - 16}):
        assert call(**bad) == rca.ERR_RANGE, bad
    for bad in ("c_k", "c_v", "c_table", "c_lengths", "c_offsets"):
        assert call(**{bad: None}) == rca.ERR_NULL, bad
    for bad in ("c_k", "c_v"):
        assert call(**{bad: M}) == rca.ERR_ALIGN, bad
    for bad in ("c_table", "c_lengths", "c_offsets"):
        assert call(**{bad: A + 2}) == rca.ERR_ALIGN, bad
    assert call(tokens=0) == rca.OK and call(c_seqs=0) == rca.OK
    assert call(tokens=0, c_k=None, c_table=None) == rca.OK


def test_append():
    for bad in ({"heads": 3}, {"heads": 65536}, {"rot": 8}, {"rot": 144}, {"positions": 63}, {"ks": 255}, {"ks": 248},
                {"ks": 260}, {"vs": 0}, {"qs": 500}, {"qs": (1 << 30) + 8}):
        assert append(**bad) == rca.ERR_RANGE, bad
    assert append(q_out=A) == rca.ERR_UNSUPPORTED
    for bad in ("k", "v", "q", "q_out"):
        assert append(**{bad: None}) == rca.ERR_NULL, bad
    for bad in ("k", "v", "q", "q_out", "rotation"):
        assert append(**{bad: M}) == rca.ERR_ALIGN, bad
    assert append(k=M, heads=0, q=None, q_out=None, qs=0) == rca.ERR_ALIGN           # no queries: none needed
    assert append(k=M, rotation=None, positions=0) == rca.ERR_ALIGN                  # no rotation: none needed
    assert append(k=M, rot=0, positions=0) == rca.ERR_ALIGN


def test_read():
    for bad in ("k", "v"):
        assert read(**{bad: None}) == rca.ERR_NULL and read(**{bad: M}) == rca.ERR_ALIGN, bad


def test_attention():
    assert attend(causal=0, window=4) == rca.ERR_UNSUPPORTED
    for bad in ({"heads": 0}, {"heads": 3}, {"heads": 65536}, {"qs": 500}, {"qs": 516}, {"tokens": 1 << 30}):
        assert attend(**bad) == rca.ERR_RANGE, bad
    for bad in ("q", "out", "ws"):
        assert attend(**{bad: None}) == rca.ERR_NULL and attend(**{bad: M}) == rca.ERR_ALIGN, bad
    assert attend(lse=A + 2) == rca.ERR_ALIGN
    size = rca.lib().rc_mxfp4_cache_attention_workspace
    assert size(10, 3, 2, 128) == 0 and size(10, 4, 0, 128) == 0 and size(10, 4, 2, 512) == 0
    assert size(10, 4, 2, 128) > 0


def test_binding_refuses():
    cpu = torch.zeros(4, 2, 64)
    kc, vc = rca.mxfp4_cache_new(2, 2, 32, 64, "cpu")
    assert kc.shape == (2, 2, 1088) and vc.shape == kc.shape and not kc.any()
    i32 = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: rca.mxfp4_cache_append(cpu, cpu, kc, vc, i32[None], i32[:1], i32),
                 lambda: rca.mxfp4_cache_read(kc, vc, i32[None], i32[:1], i32, 4, 64),
                 lambda: rca.mxfp4_cache_attention(cpu, kc, vc, i32[None], i32[:1], i32),
                 lambda: rca.mxfp4_cache_new(2, 2, 16, 64, "cpu")):
        with pytest.raises(ValueError):
            call()


@pytest.mark.gpu
def test_binding_refuses_on_the_gpu():
    dev = torch.device("cuda:0")
    x = torch.zeros(4, 2, 64, device=dev, dtype=torch.bfloat16)
    q = torch.zeros(4, 4, 64, device=dev, dtype=torch.bfloat16)
    kc, vc = rca.mxfp4_cache_new(4, 2, 32, 64, dev)
    table = torch.zeros(2, 3, dtype=torch.int32, device=dev)
    lengths, offsets = torch.tensor([2, 2], dtype=torch.int32, device=dev), torch.tensor([0, 2, 4], dtype=torch.int32, device=dev)
    rot = torch.zeros(96, 64, device=dev)
    plan = (kc, vc, table, lengths, offsets)
    bad = [
        lambda: rca.mxfp4_cache_append(x[0], x, *plan),
        lambda: rca.mxfp4_cache_append(x, x[:3], *plan),
        lambda: rca.mxfp4_cache_append(x, x.float(), *plan),
        lambda: rca.mxfp4_cache_append(x.int(), x.int(), *plan),
        lambda: rca.mxfp4_cache_append(x[:, :1], x[:, :1], *plan),                   # not the cache's heads
        lambda: rca.mxfp4_cache_append(x.transpose(0, 1).contiguous().transpose(0, 1), x, *plan),
        lambda: rca.mxfp4_cache_append(x, x, *plan, q=q[:3]),
        lambda: rca.mxfp4_cache_append(x, x, *plan, q=q.float()),
        lambda: rca.mxfp4_cache_append(x, x, *plan, q=q, q_out=q[:, :2]),
        lambda: rca.mxfp4_cache_append(x, x, *plan, rotation=rot.double()),
        lambda: rca.mxfp4_cache_append(x, x, *plan, rotation=rot[0]),
        lambda: rca.mxfp4_cache_append(x, x, kc, vc[:3], table, lengths, offsets),
        lambda: rca.mxfp4_cache_append(x, x, kc[:, :, :-1].contiguous(), vc[:, :, :-1].contiguous(), table, lengths, offsets),
        lambda: rca.mxfp4_cache_append(x, x, kc, vc, table.long(), lengths, offsets),
        lambda: rca.mxfp4_cache_append(x, x, kc, vc, table, lengths, offsets[:2]),
        lambda: rca.mxfp4_cache_append(x, x, kc, vc, table[:1], lengths, offsets),
        lambda: rca.mxfp4_cache_append(x, x, kc, vc, table[:, ::2], lengths, offsets),
        lambda: rca.mxfp4_cache_append(x, x, kc, vc, table, lengths.cpu(), offsets),
        lambda: rca.mxfp4_cache_read(*plan, 4, 64, dtype=torch.int8),
        lambda: rca.mxfp4_cache_read(*plan, 4, 64, k=x.float()),
        lambda: rca.mxfp4_cache_read(*plan, 4, 0),
        lambda: rca.mxfp4_cache_attention(q[..., ::2], *plan),
        lambda: rca.mxfp4_cache_attention(q.int(), *plan),
        lambda: rca.mxfp4_cache_attention(q, *plan, window=-1),
        lambda: rca.mxfp4_cache_attention(q, *plan, max_query=-1),
        lambda: rca.mxfp4_cache_attention(q, *plan, out=q.float()),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print("not refused:", i)
    for call, status in ((lambda: rca.mxfp4_cache_attention(q[:, :3], *plan), rca.ERR_RANGE),
                         (lambda: rca.mxfp4_cache_attention(q, *plan, causal=False, window=3), rca.ERR_UNSUPPORTED),
                         (lambda: rca.mxfp4_cache_append(x, x, *plan, q=q, rotation=rot[:95]), rca.ERR_RANGE),
                         (lambda: rca.mxfp4_cache_append(x, x, *plan, q=q, q_out=q), rca.ERR_UNSUPPORTED),
                         (lambda: rca.mxfp4_cache_append(x[:1].expand(4, 2, 64), x, *plan), rca.ERR_RANGE)):
        with pytest.raises(rca.CodecError) as e:
            call()
        assert e.value.status == status
