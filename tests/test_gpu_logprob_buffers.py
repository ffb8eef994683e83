"""One logprobs() buffer, made for many long rows with alternatives, serving calls of fewer
rows and alternatives, whose rows are shared by more workgroups: every result checked, eager and captured."""
import numpy as np
import pytest
import torch

import quantized_expert_ffn_gemv_amd as moe
import test_gpu_logprobs as gpu

pytestmark = pytest.mark.gpu
V, MOST, N_TOP = 49999, 600, 20


@pytest.fixture(scope="module")
def buffers():
    return moe.LogprobBuffers.allocate(MOST, V, N_TOP)


@pytest.fixture(scope="module")
def rows():
    rng = np.random.default_rng(21)
    return gpu.make(rng, MOST, V, True, True), rng.integers(-1, V, MOST)


@pytest.mark.parametrize("f32", [True, False])
def test_calls_of_every_size_on_one_buffer(buffers, rows, f32):
    L, tokens = rows
    if not f32:
        L = gpu.bf16_round(L)
    for T, n_top in ((MOST, 5), (1, 20), (40, 20), (1, 5), (40, 0), (1, 0), (513, 0), (7, 1), (64, 20)):
        buffers.workspace.fill_(0xFF)
        r = gpu.run(L[:T], tokens[:T], f32, n_top, buf=buffers)
        some = np.unique(np.linspace(0, T - 1, 24).astype(int))          # (the 64-bit order of 50000 elements takes a while)
        gpu.check(L[some], tokens[some], {k: v[some] if isinstance(v, np.ndarray) else v for k, v in r.items()}, n_top)


def test_captured_calls_of_two_sizes_share_a_buffer(buffers, rows):
    L, tokens = rows
    logits, tok = gpu.upload(L[:64], True), torch.from_numpy(tokens[:64].astype(np.int32)).to("cuda")
    outs = []

    def call(T, n, out):
        moe.logprobs(logits[:T], tok[:T], out[0], out[1], buffers, entropy=out[2], top_ids=out[3], top_logp=out[4])

    for T, n in ((64, 20), (1, 20), (9, 3)):
        outs.append((T, n, (torch.empty(T, device="cuda"), torch.empty(T, 2, device="cuda"), torch.empty(T, device="cuda"),
                            torch.empty(T, n, dtype=torch.int32, device="cuda"), torch.empty(T, n, device="cuda"))))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for o in outs:
            call(*o)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for o in outs:
            call(*o)
    for k in range(3):
        logits.copy_(torch.from_numpy(L[64 * k:64 * k + 64]))
        for o in outs:
            call(*o)
        torch.cuda.synchronize()
        want = [[t.clone() for t in o[2]] for o in outs]
        for o in outs:
            for t in o[2]:
                t.fill_(-3)
        buffers.workspace.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(p, q) for p, q in zip(o[2], w)), f"replay {k}, {o[0]} rows"
        host = [t.cpu().numpy() for t in outs[0][2]]
        r = dict(logp=host[0].astype(np.float64), stats=host[1].astype(np.float64), ent=host[2].astype(np.float64), ids=host[3],
                 top=host[4].astype(np.float64))
        gpu.check(L[64 * k:64 * k + 8], tokens[:8], {n: v[:8] for n, v in r.items()}, 20)
    assert int(buffers.sync.abs().sum()) == 0
