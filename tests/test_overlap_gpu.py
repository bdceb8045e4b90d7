"""The attention and expert calls are launched while the kernels before them
still run.  Whatever comes before a call in its stream, another call, a copy of
its weights, a kernel of another stream it was joined with, in a graph or not,
the results have the bits of the same calls with the device at rest between
them."""
import pytest
import torch

import gated_deltanet_linear_06_gb300 as gdn

pytestmark = pytest.mark.gpu
DEV, BF, F32, I32 = "cuda", torch.bfloat16, torch.float32, torch.int32
B, HQ, HKV, D, HID, PAGE, WIDTH, PREFIX = 24, 8, 2, 128, 1024, 16, 8, 300


class Step:
    """prep -> attention -> experts for one token of B sequences."""

    def __init__(self):
        g = torch.Generator(device=DEV).manual_seed(5)
        self.r = r = lambda *s, std=1.0: (torch.randn(*s, generator=g, device=DEV) * std).to(BF)
        self.ad = gdn.make_attn_dims(h_q=HQ, h_kv=HKV, d=D, rot=64)
        self.md = gdn.make_moe_dims(hidden=HID, inter=256, experts=16, top_k=4, shared_inter=256)
        n_pre = -(-PREFIX // PAGE)
        pages = n_pre + B * WIDTH
        self.kc, self.vc = r(pages, PAGE, HKV, D), r(pages, PAGE, HKV, D)
        self.pre = torch.arange(n_pre, dtype=I32, device=DEV)
        self.tail = (n_pre + torch.arange(B * WIDTH, device=DEV)).to(I32).view(B, WIDTH)
        self.len = (1 + torch.arange(B, device=DEV) * 5 % (WIDTH * PAGE)).to(I32)
        at = self.len.long() - 1
        self.slot = (self.tail.gather(1, (at // PAGE)[:, None])[:, 0].long() * PAGE + at % PAGE).to(I32)
        self.pos = (PREFIX + at).to(I32)
        self.inv = torch.tensor([1e4 ** (-i / 32) for i in range(32)], dtype=torch.float64, device=DEV)
        self.w = torch.ones(D, device=DEV)
        self.q, self.k, self.v = r(B, HQ, D), r(B, HKV, D), r(B, HKV, D)
        self.wr, self.gu, self.dn = r(16, HID, std=0.03), r(16, 512, HID, std=0.03), r(16, HID, 256, std=0.06)
        self.sgu, self.sdn, self.sg = r(512, HID, std=0.03), r(HID, 256, std=0.06), r(HID, std=0.03)
        self.qo = torch.empty(B, 1, HQ, D, dtype=BF, device=DEV)
        self.att = torch.empty(B, 1, HQ, D, dtype=BF, device=DEV)
        self.y = torch.empty(B, HID, dtype=BF, device=DEV)
        self.wa = torch.zeros(gdn.gdn_attn_decode_shared_workspace_bytes(self.ad, B), dtype=torch.uint8, device=DEV)
        self.wm = torch.zeros(gdn.gdn_moe_step_workspace_bytes(self.md, B), dtype=torch.uint8, device=DEV)

    def parts(self):
        return [
            lambda: gdn.gdn_attn_prep(self.ad, self.q, self.k, self.v, self.w, self.w, self.inv, None, self.pos, self.qo,
                                      self.kc, self.vc, slot=self.slot),
            lambda: gdn.gdn_attn_decode_shared(self.ad, self.qo, self.kc, self.vc, self.pre, PREFIX, self.tail, self.len,
                                               self.att, self.wa),
            lambda: gdn.gdn_moe_step(self.md, self.att.view(B, HID), self.wr, self.gu, self.dn, self.y, self.wm,
                                     w_shared_gate_up=self.sgu, w_shared_down=self.sdn, w_shared_gate=self.sg)]

    def outputs(self):
        return [t.clone() for t in (self.qo, self.kc, self.vc, self.att, self.y)]

    def inputs(self):
        return [self.q, self.k, self.v, self.gu, self.dn, self.sgu, self.sdn, self.wr]

    def alone(self):
        """The parts with the device at rest between them."""
        for part in self.parts():
            torch.cuda.synchronize()
            part()
        torch.cuda.synchronize()
        return self.outputs()


def same(a, b):
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_calls_in_a_row_on_inputs_just_written():
    s = Step()
    fresh = [[s.r(*t.shape, std=float(t.float().std())) for t in s.inputs()] for _ in range(4)]
    want = []
    for f in fresh:
        for t, n in zip(s.inputs(), f):
            t.copy_(n)
        want.append(s.alone())
    got = []
    for f in fresh:                            # copies and calls without a pause
        for t, n in zip(s.inputs(), f):
            t.copy_(n)
        for part in s.parts():
            part()
        got.append(s.outputs())
    for g, w in zip(got, want):
        same(g, w)


def test_each_call_after_itself():
    s = Step()
    want = s.alone()
    for part in s.parts():
        for _ in range(20):
            part()
    same(s.outputs(), want)


@pytest.mark.parametrize("captured", [False, True])
def test_a_call_that_joins_another_stream(captured):
    s = Step()
    src = [t.clone() for t in s.inputs()]
    want = s.alone()
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        for i, part in enumerate(s.parts()):
            # the inputs of each part are written by the other stream just before it
            side.wait_stream(main)
            with torch.cuda.stream(side):
                mine = (range(3), (), range(3, 8))[i]
                for j in mine:
                    s.inputs()[j].zero_()
                    s.inputs()[j].copy_(src[j])
            main.wait_stream(side)
            part()

    run = step
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
        stream.synchronize()
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                step()
            run = graph.replay
        for t in s.inputs() + [s.qo, s.att, s.y]:
            t.fill_(float("nan"))
        for _ in range(3):
            run()
        stream.synchronize()
    same(s.outputs(), want)


def test_captured_behind_copies_and_memory_sets():
    s = Step()
    src = [t.clone() for t in s.inputs()]
    want = s.alone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for t, n in zip(s.inputs(), src):
            t.zero_()
            t.copy_(n)
        s.y.zero_()
        for part in s.parts():
            part()
            s.wm.zero_()
    for t in s.inputs() + [s.qo, s.att, s.y]:
        t.fill_(float("nan"))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    same(s.outputs(), want)
