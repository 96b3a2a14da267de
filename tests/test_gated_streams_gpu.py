"""Who may free what while another stream still works: 4-bit weights that are made from temporaries,
and ones that are dropped behind a call."""
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
U8 = torch.uint8


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from tensor_transformer_mlp_03_amd import _lib as L
    L.lib()


@pytest.fixture(autouse=True)
def _announce(request):
    print(f"[case] {request.node.name}", flush=True)
    sys.stdout.flush()


class Case:
    """A weight of 4096 x 4096, its product on the current stream, and another stream with some tenths of a
    second of work before it."""

    def __init__(self):
        from tensor_transformer_mlp_03_amd.gated import Fp4Linear
        gen = torch.Generator("cuda").manual_seed(6)
        self.W = torch.randn(4096, 4096, device="cuda", generator=gen).bfloat16()
        self.codes = torch.randint(0, 256, (4096, 2048), dtype=U8, device="cuda", generator=gen)
        self.scales = torch.randint(120, 130, (4096, 128), dtype=U8, device="cuda", generator=gen)
        self.X = torch.randn(3, 4096, device="cuda", generator=gen).bfloat16()
        self.want, self.from_w, self.Y = (torch.empty(3, 4096, device="cuda") for _ in range(3))
        Fp4Linear(self.codes, self.scales).forward(self.X, self.want)
        Fp4Linear.from_weight(self.W).forward(self.X, self.from_w)
        self.busy = [torch.randn(8192, 8192, device="cuda", generator=gen).bfloat16() for _ in range(2)]
        torch.mm(*self.busy)
        for _ in range(8):  # one that does not share a hardware queue with the current stream, which would wait for it
            self.stream = torch.cuda.Stream()
            self.work(40)
            self.X.add_(0)
            torch.cuda.current_stream().synchronize()
            if not self.stream.query():
                break
        self.fill(2)
        torch.cuda.synchronize()

    def work(self, n=100):
        self.stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(self.stream):
            out = torch.empty_like(self.busy[0])
            for _ in range(n):
                torch.mm(*self.busy, out=out)

    def fill(self, n):
        """n tensors of every size in play, which would lie where freed ones were."""
        sizes = [self.codes.numel(), self.scales.numel(), 2 * self.W.numel(), 4096 * 32 * 68]
        return [torch.full((k,), 0x91, dtype=U8, device="cuda") for k in sizes for _ in range(n)]

    def holds(self, want):
        """After the call: fills the memory that is free, and compares what the other stream makes."""
        fill = self.fill(3)  # two of each size are there already: a third is what was freed, or new
        torch.cuda.current_stream().synchronize()
        self.stream.synchronize()
        assert torch.equal(self.Y, want) and fill


@pytest.mark.parametrize("handle", [False, True])
def test_fp4_weight_from_temporaries(handle):
    from tensor_transformer_mlp_03_amd.gated import Fp4Linear
    c = Case()
    codes, scales = c.codes.clone(), c.scales.clone()
    c.work()
    s = c.stream.cuda_stream if handle else c.stream
    lin = Fp4Linear(codes, scales, stream=s)
    del codes, scales
    lin.forward(c.X, c.Y, stream=s)
    c.holds(c.want)


def test_fp4_weight_from_a_temporary_bf16_weight():
    from tensor_transformer_mlp_03_amd.gated import Fp4Linear
    c = Case()
    W = c.W.clone()
    c.work()
    lin = Fp4Linear.from_weight(W, stream=c.stream)
    del W
    lin.forward(c.X, c.Y, stream=c.stream)
    c.holds(c.from_w)


@pytest.mark.parametrize("current", [False, True])
def test_fp4_weight_dropped_behind_a_call(current):
    from tensor_transformer_mlp_03_amd.gated import Fp4Linear
    c = Case()
    lin = Fp4Linear(c.codes, c.scales)
    c.work()
    if current:
        with torch.cuda.stream(c.stream):
            lin.forward(c.X, c.Y)
    else:
        lin.forward(c.X, c.Y, stream=c.stream)
    del lin
    c.holds(c.want)


def test_fp4_weight_with_pinned_scales():
    from tensor_transformer_mlp_03_amd.gated import Fp4Linear
    c = Case()
    codes, scales = c.codes.clone(), c.scales.cpu().pin_memory()
    c.work()
    lin = Fp4Linear(codes, scales, stream=c.stream)
    del codes, scales
    lin.forward(c.X, c.Y, stream=c.stream)
    pinned = [torch.full((4096, 128), 0x91, dtype=U8).pin_memory() for _ in range(4)]
    c.holds(c.want)
    del pinned
