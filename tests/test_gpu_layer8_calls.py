"""Calls of the attention layer in 8 bits from the side of their caller: streams, devices, outputs that lie beside or over
their inputs."""
import pytest
import torch

pytestmark = pytest.mark.gpu
FP8, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
T, HQ, HKV, DIM, PAGE, PAGES, HIDDEN = 23, 6, 2, 128, 32, 9, 256


class Layer:
    """One layer's tensors: two requests of 11 and 12 new tokens in front of nothing."""

    def __init__(self, B, kind, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        i32 = dict(dtype=torch.int32, device="cuda")
        self.B, self.x = B, rnd(T, HIDDEN)
        self.w = B.int8_quantize(rnd((HQ + 2 * HKV) * DIM, HIDDEN))
        self.o = B.int8_quantize(rnd(HIDDEN, HQ * DIM))
        self.k, self.v = (torch.zeros(PAGES, HKV, PAGE, DIM, dtype=torch.uint8, device="cuda").view(kind) for _ in range(2))
        self.ks, self.vs = (torch.zeros(PAGES, HKV, PAGE // 16, dtype=torch.uint8, device="cuda").view(E8M0) for _ in range(2))
        self.table = torch.tensor([[7], [2]], **i32)
        self.q_start, self.lens = torch.tensor([0, 11, 23], **i32), torch.tensor([11, 12], **i32)
        self.positions = torch.cat([torch.arange(11, **i32), torch.arange(12, **i32)])
        self.slots = self.positions.long() + torch.where(torch.arange(T, device="cuda") < 11, 7, 2) * PAGE
        self.rotation = B.rotary_table(DIM)
        self.ws = B.paged_attention_workspace(T, 2, HQ, HKV, DIM, 12, 32)

    def __call__(self):
        B, nq, nk = self.B, HQ * DIM, HKV * DIM
        y = B.int8_linear(self.x, *self.w)
        q = B.paged_kv_append(y[:, nq:nq + nk], y[:, nq + nk:], self.positions, self.slots, self.k, self.v, rotation=self.rotation,
                              k_scale=self.ks, v_scale=self.vs, q=y[:, :nq])
        a = B.paged_attention_blocks(q, self.k, self.v, self.ks, self.vs, self.table, self.q_start, self.lens, 12, 32,
                                     workspace=self.ws)
        return B.int8_linear(a, *self.o)


def test_two_streams_at_once(gpu_lib):
    """Two layers in flight side by side give what each gives alone."""
    layers = [Layer(gpu_lib, kind, i) for i, kind in enumerate((FP8, torch.int8))]
    alone = [layer() for layer in layers]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in layers], [[], []]
    for _ in range(8):
        for i, layer in enumerate(layers):
            with torch.cuda.stream(streams[i]):
                got[i].append(layer())
    torch.cuda.synchronize()
    for want, all_ in zip(alone, got):
        assert want.float().abs().max() > 0
        for y in all_:
            assert torch.equal(y, want)


def test_tensors_of_another_gpu_than_the_current_one(gpu_lib, monkeypatch):
    layer = Layer(gpu_lib, FP8, 3)
    y = torch.zeros(T, (HQ + 2 * HKV) * DIM, dtype=torch.bfloat16, device="cuda")
    q, k = y[:, :HQ * DIM], y[:, :HKV * DIM]
    codes, scale = gpu_lib.int8_quantize(layer.x)
    monkeypatch.setattr(gpu_lib, "_current_device", lambda: layer.x.get_device() + 1)
    for call in (lambda: gpu_lib.rotary(q, layer.positions, layer.rotation, DIM),
                 lambda: gpu_lib.paged_kv_append(k, k, layer.positions, layer.slots, layer.k, layer.v, k_scale=layer.ks, v_scale=layer.vs),
                 lambda: gpu_lib.paged_attention_blocks(q, layer.k, layer.v, layer.ks, layer.vs, layer.table, layer.q_start,
                                                        layer.lens, 12, 32, workspace=layer.ws),
                 lambda: gpu_lib.int8_quantize(layer.x), lambda: gpu_lib.gemm_w8a8(codes, scale, *layer.w),
                 lambda: gpu_lib.int8_linear(layer.x, *layer.w)):
        with pytest.raises(gpu_lib.NVFP4Error, match="the current one"):
            call()


@pytest.mark.parametrize("m", [1, 37, 300])
def test_int8_outputs_beside_and_over_inputs(gpu_lib, m):
    """An output may be other columns of the input's matrix; one that shares elements with an input is refused."""
    g = torch.Generator(device="cuda").manual_seed(m)
    both = torch.randn(m, 512, generator=g, device="cuda").to(torch.bfloat16)
    w, s = gpu_lib.int8_quantize(torch.randn(256, 256, generator=g, device="cuda").to(torch.bfloat16))
    x = both[:, :256]
    want = gpu_lib.int8_linear(x.clone(), w, s)
    assert torch.equal(gpu_lib.int8_linear(x, w, s, out=both[:, 256:]), want)
    codes, scales = gpu_lib.int8_quantize(x)
    for call in (lambda: gpu_lib.int8_linear(x, w, s, out=both[:, 128:384]), lambda: gpu_lib.int8_linear(x, w, s, out=both[:, :256]),
                 lambda: gpu_lib.int8_linear(x, w, s, out_dtype=torch.float32, out=both.view(torch.float32)),
                 lambda: gpu_lib.gemm_w8a8(codes, scales, w[:128], s[:128], out=codes.view(torch.bfloat16))):
        with pytest.raises(gpu_lib.NVFP4Error, match="overlap"):
            call()
