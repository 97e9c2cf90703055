"""The operators around the draft and the verify on streams forked from and joined to
the one that makes their inputs and reads their outputs, run and captured."""
import pytest
import torch

from block_diffusion_speculative_fusion_gb300 import api

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _built():
    from block_diffusion_speculative_fusion_gb300 import build
    build.build()
    api.lib()


def test_forked_streams_run_and_captured():
    B, R, V, T, K, N, page, pages = 4, 5, 30011, 40, 2048, 640, 16, 64
    g = torch.Generator().manual_seed(1)
    n = 5
    z = torch.randn((n, B, R, V), generator=g).to(torch.bfloat16).to(DEV)
    hist = torch.randint(0, V, (n, B, 500), generator=g).to(DEV)
    x = torch.randn((n, T, K), generator=g).to(torch.bfloat16).to(DEV)
    length = torch.randint(1, page * pages, (n, B), generator=g).to(torch.int32).to(DEV)
    w, ws = api.fp8_quant(torch.randn((N, K), generator=g).to(torch.bfloat16).to(DEV), block_rows=128)
    hl = torch.full((B,), 500, dtype=torch.int32, device=DEV)
    rep = torch.full((B,), 1.25, device=DEV)
    nd = torch.full((B,), R - 1, dtype=torch.int32, device=DEV)
    zero = torch.zeros(B, dtype=torch.int32, device=DEV)
    buf = dict(z=torch.empty_like(z[0]), h=torch.empty_like(hist[0]), x=torch.empty_like(x[0]),
               q=torch.empty((T, K), dtype=torch.float8_e4m3fn, device=DEV), s=torch.empty((T, K // 128), device=DEV),
               len=torch.empty_like(length[0]), free=torch.empty(B * pages, dtype=torch.int32, device=DEV),
               table=torch.empty((B, pages), dtype=torch.int32, device=DEV))
    out = dict(z=torch.empty_like(z[0]), y=torch.empty((T, N), dtype=torch.bfloat16, device=DEV),
               pg=dict(n_pages=torch.empty_like(zero), n_free=zero[:1].clone(), short=torch.empty(B, dtype=torch.uint8, device=DEV)),
               sm=torch.empty(B * page * pages, dtype=torch.int64, device=DEV))
    rows_max = B * page * pages
    cand = torch.randint(0, V, (B, R), generator=g).to(DEV)
    keep = torch.empty((n, B), dtype=torch.int64, device=DEV)
    ys, sms = torch.empty((n, *out["y"].shape), dtype=torch.bfloat16, device=DEV), torch.empty((n, rows_max), dtype=torch.int64, device=DEV)
    side = [torch.cuda.Stream() for _ in range(3)]
    nf = torch.full((1,), B * pages, dtype=torch.int32, device=DEV)

    def run(fork):
        main = torch.cuda.current_stream()
        for i in range(n):
            # made on the main stream by kernels
            buf["z"].copy_(z[i]).mul_(2)
            buf["h"].copy_(hist[i])
            buf["x"].copy_(x[i])
            buf["len"].copy_(length[i])
            buf["table"].fill_(-1)
            buf["free"].copy_(torch.arange(B * pages, dtype=torch.int32, device=DEV))
            streams = side if fork else [main] * 3
            for st in side if fork else []:
                st.wait_stream(main)
            with torch.cuda.stream(streams[0]):
                api.logits_rules(buf["z"], cand=cand, n_draft=nd, hist=buf["h"], hist_len=hl, repetition=rep, out=out["z"])
            with torch.cuda.stream(streams[1]):
                api.fp8_quant(buf["x"], q=buf["q"], scale=buf["s"])
                api.fp8_gemm(buf["q"], buf["s"], w, ws, out=out["y"])
            with torch.cuda.stream(streams[2]):
                api.pages_resize(buf["len"], buf["table"], zero, buf["free"], nf, page, out=out["pg"])
                api.slot_map(zero, buf["len"], buf["table"], page, B * pages, rows_max, out=dict(slots=out["sm"]))
            for st in side if fork else []:
                main.wait_stream(st)
            # read on the main stream
            keep[i] = api.verify_greedy(out["z"], cand, nd)["bonus"]
            ys[i].copy_(out["y"])
            sms[i].copy_(out["sm"])

    run(False)
    torch.cuda.synchronize()
    want = [t.clone() for t in (keep, ys, sms)]
    assert bool((want[2] >= 0).any()) and not torch.equal(want[1][0], want[1][1])
    graph = torch.cuda.CUDAGraph()
    for t in (keep, ys, sms):
        t.zero_()
    run(True)
    torch.cuda.synchronize()
    for a, b in zip((keep, ys, sms), want):
        assert torch.equal(a, b)
    with torch.cuda.graph(graph):
        run(True)
    for _ in range(3):
        for t in (keep, ys, sms):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((keep, ys, sms), want):
            assert torch.equal(a, b)
