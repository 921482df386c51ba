"""The three kernels of a call over shared prefixes overlap each other's starts:
calls one behind the other in one workspace, each with another plan, and nothing
between them, eagerly and replayed, give what each gives by itself."""
import pytest
import torch

from exact_attention_94_gb300 import _lib, ops
from tests.test_decode_shared_gpu import call, i32, make

pytestmark = pytest.mark.gpu

BATCHES = [([(100, [120, 130, 300])], 1, 8, 2, 128), ([(40, [90, 50])] * 6, 4, 8, 2, 64), ([(777, [800, 790, 1, 0])], 1, 32, 8, 128),
           ([(0, [5]), (300, [301] * 40), (16, [17, 16])], 1, 8, 8, 64), ([(0, [0, 0]), (7, [0, 120])], 2, 16, 1, 128)]


@pytest.mark.parametrize("replayed", [False, True])
def test_one_behind_the_other(replayed):
    batches = [make(*b, 16, seed=i) for i, b in enumerate(BATCHES)]
    alone = []
    for m in batches:
        alone.append(call(m))
        torch.cuda.synchronize()
    size = max(_lib.load().fa_decode_shared_workspace_bytes(len(m["lens"]), *m["q"].shape[1:3], m["k"].shape[2], m["q"].shape[3],
                                                            len(m["shared"]), 0) for m in batches)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    args = [[m[x].cuda() for x in "qkv"] + [i32(m[x]) for x in ("table", "lens", "starts", "shared")] + [max(m["lens"])]
            for m in batches]
    order = [(5 * i + i // 7) % len(batches) for i in range(60)]

    def run():
        return [ops.decode_paged_shared(*args[i], workspace=ws) for i in order]
    if replayed:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run()
        for _ in range(5):
            graph.replay()
    else:
        got = run()
    torch.cuda.synchronize()
    for i, (o, lse) in zip(order, got):
        assert torch.equal(o, alone[i][0]) and torch.equal(lse, alone[i][1]), i
    assert ops.device_error() == 0
