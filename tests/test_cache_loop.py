"""The loop that Cache8's documentation gives, run as written against stand-ins of the
calls: which lengths each layer's calls are handed.  (Run on the kernels in
test_gpu_cache_contract.py.)"""
import re
import textwrap
import types

import pytest

from block_top_sparse_b200 import ops

torch = pytest.importorskip("torch")


def documented_loop():
    code = re.search(r"::\n\n((?:        .*\n|\n)+)", ops.Cache8.__doc__ or "")
    assert code, "Cache8 shows no loop"
    return compile(textwrap.dedent(code.group(1)), "Cache8", "exec")


def test_every_layer_sees_the_lengths_of_the_step():
    s, keep = 64, 2
    B, H, d, n = 4, 2, 8, 5
    seen = {"append": [], "decode": [], "evict": []}

    def decode(dims, cache, last, q, weight_in, weight_out):
        seen["decode"].append(last.tolist())
        assert q.shape == (B, H, d) and q.is_contiguous() and last.dtype == torch.int32
        assert weight_in is weight_out is cache.weight
        # every sequence's newest token attends
        assert [float(x) for x in q[:, 0, 0]][:2] == [float(cache.q[0, 0, 4, 0]), float(cache.q[1, 0, 0, 0])]
        return q, None, None

    def evict(dims, cache, cache_len, keep, weight, sink=0, recent=0, weight_out=None):
        seen["evict"].append(cache_len.tolist())
        assert sink + recent <= keep
        whole = cache_len // s
        return None, torch.where(whole > keep, keep * s + cache_len % s, cache_len).int()

    fake = types.SimpleNamespace(
        rope_axes=lambda dims, pos, sections, q, k: (q, k),
        cache_append=lambda dims, cache, cache_len, k, v, n_new: seen["append"].append((cache_len.tolist(), n_new.tolist())),
        cache_decode=decode, cache_evict=evict)
    caches = [types.SimpleNamespace(q=torch.rand(B, H, n, d), weight=object()) for _ in range(3)]
    cache_len = torch.tensor([200, 63, -1, 100], dtype=torch.int32)
    env = dict(ops=fake, torch=torch, dims=None, dims_n=None, pos=None, sections=None, caches=caches, x=None, keep=keep,
               sink=1, recent=1, weights=[c.weight for c in caches], cache_len=cache_len,
               n_new=torch.tensor([5, 1, 0, 0], dtype=torch.int32), rows=torch.arange(B),
               layers=[(lambda x, c=c: (c.q, c.q, c.q)) for c in caches])
    exec(documented_loop(), env)
    assert seen["append"] == [([200, 63, -1, 100], [5, 1, 0, 0])] * 3
    assert seen["decode"] == [[204, 63, -1, -1]] * 3     # a sequence without new tokens attends nothing
    assert seen["evict"] == [[205, 64, -1, 100]] * 3     # the lengths from before any layer's eviction
    assert env["cache_len"] is cache_len and cache_len.tolist() == [2 * s + 205 % s, 64, -1, 100]
