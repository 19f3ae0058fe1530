"""Training operators called from several host threads at once, each on a stream of
its own and with other sizes: the results are those of calls one after another."""
import threading

import pytest
import torch

import top_routing_expert_gb300 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    moe.load_library()


def _block_job(T, H, k):
    g = torch.Generator(device=DEV).manual_seed(H + k)
    bf = lambda *n: torch.randn(n, generator=g, device=DEV).to(torch.bfloat16)
    h, y, go, gx = bf(T, H), bf(T * k, H), bf(T, H), bf(T, H)
    dest = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32).view(T, k)
    w = torch.rand(T, k, generator=g, device=DEV)
    weight = torch.rand(H, generator=g, device=DEV)
    cfg, ws = moe.BlockConfig.make(), moe.BlockWorkspace(T, H)

    def run():
        out = [torch.empty_like(h), torch.empty_like(y), torch.empty(T, k, device=DEV),
               torch.empty(H, device=DEV), torch.empty(H, device=DEV)]
        moe.moe_block_norm_bwd(cfg, h, y, go, out[0], out[1], grad_xn=gx, dest_row=dest, topk_w=w,
                               post_weight=weight, pre_weight=weight, grad_topk_w=out[2],
                               grad_post=out[3], grad_pre=out[4], ws=ws)
        return out
    return run


def _product_job(E, rows, K, N):
    g = torch.Generator(device=DEV).manual_seed(E)
    bf = lambda *n: torch.randn(n, generator=g, device=DEV).to(torch.bfloat16)
    x, y, W = bf(rows, K), bf(rows, N), bf(E, K, N)
    offsets = torch.linspace(0, rows, E + 1).to(torch.int32).to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run():
        out = [torch.empty(rows, N, dtype=torch.bfloat16, device=DEV), torch.empty(E, K, N, device=DEV)]
        moe.moe_expert_gemm(x, offsets, W, out[0], dev_status=status)
        moe.moe_expert_wgrad(x, y, offsets, out[1], dev_status=status)
        return out
    return run


def test_threads():
    jobs = [_block_job(200, 4096, 2), _block_job(150, 4096, 8), _block_job(300, 2816, 1),
            _product_job(3, 500, 128, 192), _product_job(256, 700, 64, 64), _product_job(1, 4096, 256, 128)]
    want = [j() for j in jobs]
    torch.cuda.synchronize()
    wrong = []

    def work(n):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(25):
                    got = jobs[n]()
                    stream.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[n])):
                        wrong.append(n)
        except Exception as e:
            wrong.append((n, repr(e)))

    threads = [threading.Thread(target=work, args=(n,)) for n in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
