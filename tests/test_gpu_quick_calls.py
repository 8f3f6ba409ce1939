"""The host-bound calls through the extension and through the Python checks:
one result, one set of refusals."""

import pytest
import torch

import paged_kv_cache_386_b200 as pkv
from tests.gpu_helpers import bits


@pytest.fixture(scope="module")
def ext():
    from paged_kv_cache_386_b200 import build

    build.build()
    return pkv._quick()


@pytest.fixture
def checked(monkeypatch):
    """Calls go through the Python checks alone."""
    def run(f):
        with monkeypatch.context() as m:
            m.setattr(pkv, "_ext", False)
            m.setattr(pkv, "_quick", lambda: False)
            return f()
    return run


def test_not_for_cpu_tensors(ext):
    k, slots, table = torch.zeros(2, 2, 64), torch.zeros(2, dtype=torch.int64), torch.zeros(4, 64)
    cache, (kv, sc) = torch.zeros(3, 2, 16, 64), pkv.fp8_cache(3, 2, 64, device="cpu")
    bt, cl = torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    assert ext.append_rope(k, k, slots, table, slots, cache, cache, None, None, False, False) is NotImplemented
    assert ext.append_rope(k, k, slots, table, slots, kv, sc, k, k, True, True) is NotImplemented
    assert ext.append_fp8(k, k, slots, kv, sc) is NotImplemented
    assert ext.decode_fp8(k.half(), kv, sc, bt, cl, 0.1, None, None) is NotImplemented
    # Nothing that is no tensor, and no wrong count of arguments, is read either.
    for f, n in ((ext.append_rope, 11), (ext.append_fp8, 5), (ext.decode_fp8, 8)):
        for args in ((None,) * n, (1,) * n, (k,) * (n - 1), ()):
            assert f(*args) is NotImplemented


class Case:
    def __init__(self, d=128, n_q=8, n_kv=2, n=37, dtype=torch.bfloat16, seed=0):
        g = torch.Generator().manual_seed(seed)
        rows = torch.randn((n, (n_q + 2 * n_kv) * d), generator=g).to(dtype).cuda()
        self.q, self.k, self.v = (x.unflatten(1, (-1, d)) for x in rows.split((n_q * d, n_kv * d, n_kv * d), 1))
        self.pos, self.slots = torch.arange(100, 100 + n).cuda(), torch.arange(5, 5 + n).cuda()
        self.table = pkv.rotary_table(256, d)
        self.kc, self.vc = (torch.randn((4, n_kv, 16, d), generator=g).to(dtype).cuda() for _ in range(2))
        self.kv, self.sc = pkv.fp8_cache(4, n_kv, d)
        self.bt = torch.arange(4, dtype=torch.int32).cuda()[None]
        self.cl = torch.tensor([5 + n], dtype=torch.int32).cuda()

    def rope(self, **kw):
        return pkv.paged_kv_append_rope(self.k, self.v, self.pos, self.table, self.slots, self.kc, self.vc, **kw)

    def rope_fp8(self, **kw):
        return pkv.paged_kv_append_rope_fp8(self.k, self.v, self.pos, self.table, self.slots, self.kv, self.sc, **kw)

    def append(self, **kw):
        return pkv.paged_kv_append_fp8(self.k, self.v, self.slots, self.kv, self.sc, **kw)

    def decode(self, q, **kw):
        return pkv.paged_attention_decode_fp8(q, self.kv, self.sc, self.bt, self.cl, 0.1, **kw)

    def everything(self):
        out = [self.rope(q=self.q, interleaved=True)]
        none = [self.rope(), self.append()]
        out += [self.rope_fp8(q=self.q), self.rope_fp8(q=self.q, q_out=self.q)]
        assert none == [None, None] and out[-1] is self.q
        if self.q.dtype != torch.float32:
            q = out[1][-3:].contiguous()
            ws = pkv.new_workspace(pkv.paged_attention_fp8_workspace_size(1, len(q), q.shape[1], self.kv.shape[1],
                                                                          q.shape[2], device="cuda"))
            o = torch.empty_like(q)[None]
            assert self.decode(q[None], out=o) is o
            out += [o, self.decode(q[None], workspace=ws), self.decode(q[:1])]
        return [bits(x.contiguous()) for x in (*out, self.kc, self.vc, self.kv.view(torch.uint8), self.sc)]


@pytest.mark.gpu
@pytest.mark.parametrize("n_q,n_kv,d,dtype", [(8, 2, 128, torch.bfloat16), (3, 3, 64, torch.float16),
                                              (4, 1, 64, torch.float32), (1, 1, 128, torch.bfloat16)])
@pytest.mark.parametrize("n", [1, 37])
def test_one_result_either_way(ext, checked, n, n_q, n_kv, d, dtype):
    a, b = (Case(d, n_q, n_kv, n, dtype) for _ in range(2))
    for got, want in zip(a.everything(), checked(b.everything), strict=True):
        assert got.shape == want.shape and torch.equal(got, want)


@pytest.mark.gpu
def test_the_plain_case_is_taken_and_a_refused_one_is_not(ext):
    c = Case()
    args = (c.k, c.v, c.pos, c.table, c.slots)
    assert ext.append_rope(*args, c.kc, c.vc, None, None, False, False) is None
    assert ext.append_rope(*args, c.kv, c.sc, c.q, c.q, False, True) is c.q
    assert ext.append_fp8(c.k, c.v, c.slots, c.kv, c.sc) is None
    q = c.q[:1].contiguous()
    assert ext.decode_fp8(q, c.kv, c.sc, c.bt, c.cl, 0.1, None, None).shape == q.shape
    before = [x.clone() for x in (c.kc, c.vc, c.kv.view(torch.uint8), c.sc)]
    for bad in ((c.k.half(), *args[1:], c.kc, c.vc), (c.k, c.v[:5], *args[2:], c.kc, c.vc),
                (c.k, c.v, c.pos.int(), *args[3:], c.kc, c.vc), (c.k, c.v, c.pos, c.table.half(), c.slots, c.kc, c.vc),
                (*args[:4], c.slots[:5], c.kc, c.vc), (*args, c.kc, c.vc[:2]), (*args, c.kc[:, :1], c.vc[:, :1]),
                (*args, c.kc.transpose(1, 2), c.vc.transpose(1, 2)), (*args[:4], c.slots.cpu(), c.kc, c.vc),
                (c.k.transpose(1, 2).contiguous().transpose(1, 2), *args[1:], c.kc, c.vc),
                (c.k, c.v, c.pos, c.table[:, :7].contiguous(), c.slots, c.kc, c.vc)):
        assert ext.append_rope(*bad, None, None, False, False) is NotImplemented
        with pytest.raises((ValueError, pkv.PagedKVError)):
            pkv.paged_kv_append_rope(*bad)
    for q_bad, out in ((c.q.half(), None), (c.q[:5], None), (c.q, c.q[:5]), (c.q, c.q.half()), (c.q[..., :64], None),
                       (None, c.q)):
        assert ext.append_rope(*args, c.kv, c.sc, q_bad, out, False, True) is NotImplemented
        with pytest.raises(ValueError):
            c.rope_fp8(q=q_bad, q_out=out)
    for bad in ((c.k, c.v, c.slots, c.kv.view(torch.uint8), c.sc), (c.k, c.v, c.slots, c.kv, c.sc[:2]),
                (c.k, c.v, c.slots, c.kv.transpose(0, 1), c.sc), (c.k, c.v, c.slots, c.kv, c.sc.half())):
        assert ext.append_fp8(*bad) is NotImplemented
        with pytest.raises(ValueError):
            pkv.paged_kv_append_fp8(*bad)
    for bad in ((q.float(), c.kv, c.sc, c.bt, c.cl), (q, c.kv, c.sc, c.bt.long(), c.cl), (q, c.kv, c.sc, c.bt, c.bt),
                (q, c.kv, c.sc, c.bt[:, ::2], c.cl), (q[0], c.kv, c.sc, c.bt, c.cl), (q.cpu(), c.kv, c.sc, c.bt, c.cl)):
        assert ext.decode_fp8(*bad, 0.1, None, None) is NotImplemented
        with pytest.raises((ValueError, pkv.PagedKVError)):
            pkv.paged_attention_decode_fp8(*bad, 0.1)
    small = torch.zeros(256, dtype=torch.uint8, device="cuda")
    assert ext.decode_fp8(q, c.kv, c.sc, c.bt, c.cl, 0.1, None, small) is NotImplemented
    assert ext.decode_fp8(q, c.kv, c.sc, c.bt, c.cl, 0.1, q.half(), None) is NotImplemented
    torch.cuda.synchronize()
    for x, y in zip(before, (c.kc, c.vc, c.kv.view(torch.uint8), c.sc)):
        assert torch.equal(bits(x), bits(y))


@pytest.mark.gpu
def test_current_stream_and_graph(ext):
    """The work of a call is on the current stream, under capture too."""
    want = Case().everything()
    c, side = Case(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = c.everything()
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want, strict=True))

    c = Case()
    q, kv0, sc0 = c.q.clone(), c.kv.clone(), c.sc.clone()
    c.rope_fp8(q=c.q)
    c.kv.copy_(kv0), c.sc.copy_(sc0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q2 = c.rope_fp8(q=c.q)
        out = c.decode(q2[-1:])
    assert torch.equal(c.kv.view(torch.uint8), kv0.view(torch.uint8))  # captured, not run
    graph.replay()
    torch.cuda.synchronize()
    e = Case()
    want_q = e.rope_fp8(q=q)
    assert torch.equal(bits(q2), bits(want_q)) and torch.equal(bits(out), bits(e.decode(want_q[-1:])))
    assert torch.equal(c.kv.view(torch.uint8), e.kv.view(torch.uint8)) and torch.equal(c.sc, e.sc)


@pytest.mark.gpu
def test_threads_with_a_stream_each(ext):
    """Calls release the interpreter while they launch: threads do not disturb one another."""
    from concurrent.futures import ThreadPoolExecutor

    want = {seed: Case(seed=seed).everything() for seed in range(4)}
    cases = {seed: [Case(seed=seed) for _ in range(8)] for seed in want}
    torch.cuda.synchronize()

    def work(seed):
        with torch.cuda.stream(torch.cuda.Stream()):
            got = [c.everything() for c in cases[seed]]
            torch.cuda.current_stream().synchronize()
        return got

    with ThreadPoolExecutor(4) as pool:
        for seed, results in zip(want, pool.map(work, want), strict=True):
            for got in results:
                assert all(torch.equal(x, y) for x, y in zip(got, want[seed], strict=True))


@pytest.mark.gpu
def test_one_row_for_all_tokens(ext, checked):
    """Inputs whose tokens are one broadcast row; an output may not be one."""
    a, b = Case(), Case()
    for c in (a, b):
        c.k, c.v, c.q = (x[:1].expand(len(c.slots), -1, -1) for x in (c.k, c.v, c.q))
    got, want = a.rope_fp8(q=a.q), checked(lambda: b.rope_fp8(q=b.q))
    assert torch.equal(bits(got), bits(want)) and torch.equal(a.sc, b.sc)
    assert torch.equal(a.kv.view(torch.uint8), b.kv.view(torch.uint8))
    with pytest.raises(pkv.PagedKVError):
        a.rope_fp8(q=a.q, q_out=a.q)
