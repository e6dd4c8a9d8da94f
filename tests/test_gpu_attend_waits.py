"""The waits of the attention kernels are about their own work, however long what is ahead of
them on the stream takes."""
import time

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from paged_kv_gather_gb300.build import build  # noqa: E402

build()
from paged_kv_gather_gb300 import kvx  # noqa: E402
from paged_kv_gather_gb300 import workloads as wl  # noqa: E402
from tests.cache_common import Cache  # noqa: E402


class SlowLoad:
    """A load by one warp with one 16-byte unit a lane in flight, launched to overlap: it lets
    the next kernel of its stream start at once and runs on beside it."""

    PAGE, TOKEN = 16, 1024

    def __init__(self, ctx, tokens, parts):
        total = tokens * parts
        self.tokens, self.parts = tokens, parts
        n = total // self.PAGE
        self.pages = torch.zeros((1, 1, n, self.PAGE, self.TOKEN), dtype=torch.uint8,
                                 device="cuda")
        self.table = torch.arange(n, dtype=torch.int32, device="cuda")
        self.host = kvx.HostBuffer(tokens * self.TOKEN)
        self.host.array[:] = 7
        reqs = kvx.requests_array([(self.table.data_ptr(), None, total)])
        # Every chunk reads the same host memory into pages of its own.
        chunks = kvx.chunks_array([wl.ChunkSpec(0, i * tokens, tokens, 0, 1, wl.LAYER_MAJOR, 0)
                                   for i in range(parts)], self.host.ptr)
        cfg = kvx.kvx_default_launch_cfg(ctx, kvx.KVX_OP_LOAD)
        cfg.sm_cap, cfg.ctas_per_sm, cfg.threads = 1, 1, 32
        cfg.unroll, cfg.batch, cfg.overlap = 1, 1, 1
        torch.cuda.synchronize()
        self.plan = kvx.kvx_plan_create(ctx, kvx.KVX_OP_LOAD,
                                        kvx.Pool.from_tensor(self.pages, self.PAGE), reqs, chunks,
                                        cfg=cfg)

    def launch(self, stream):
        kvx.kvx_plan_launch(self.plan, stream.cuda_stream)

    def close(self):
        torch.cuda.synchronize()
        kvx.kvx_plan_destroy(self.plan)
        self.host.close()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("new", [1, 200])
def test_a_long_transfer_ahead(new, kv):
    """Attention that starts beside a transfer of more than a second, the limit of its own
    waits, gives what it gives on an idle GPU."""
    ctx = kvx.kvx_create(0)
    cache = Cache([900, 300], 2, 128, 16, kv)
    q = torch.randn((2 * new, 8, 128), device="cuda").bfloat16()
    plan = kvx.kvx_attn_plan_create(ctx, cache.kvx_pool, cache.requests(), [new, new],
                                    kvx.attn_config(8, 2, 128, "bf16", kv))
    want, out = torch.empty_like(q), torch.zeros_like(q)
    kvx.kvx_attend(plan, 1, q.data_ptr(), want.data_ptr())
    torch.cuda.synchronize()

    stream = torch.cuda.Stream()
    short = SlowLoad(ctx, 2048, 1)
    short.launch(stream)
    torch.cuda.synchronize()
    t = time.perf_counter()
    short.launch(stream)
    torch.cuda.synchronize()
    each = time.perf_counter() - t
    short.close()
    load = SlowLoad(ctx, 2048, max(1, min(8192, int(1.6 / each) + 1)))
    torch.cuda.synchronize()
    t = time.perf_counter()
    load.launch(stream)
    kvx.kvx_attend(plan, 1, q.data_ptr(), out.data_ptr(), stream=stream.cuda_stream)
    torch.cuda.synchronize()
    took = time.perf_counter() - t
    assert took > 1.2
    assert kvx.kvx_get_status(ctx) == 0
    assert torch.equal(out, want) and bool((load.pages == 7).all())
    load.close()
    kvx.kvx_attn_plan_destroy(plan)
    kvx.kvx_destroy(ctx)
