"""The benchmark's check covers the outputs that its timed calls have written,
also where there are fewer calls than input sets (host logic, no GPU)."""
import os
import sys

import torch

import oracle
import synth

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bench  # noqa: E402


class Calls:
    """Stands for the library: each call writes the oracle's outputs."""

    def __init__(self, o):
        self.o, self.case, self.made = o, None, 0

    def __getattr__(self, name):  # the other rules, which are not called
        return None

    def spec_verify_greedy(self, *args):
        out = self.case.outputs[self.made % self.case.sets]
        assert args[6].value == out["tok"].data_ptr()
        out["tok"].copy_(torch.from_numpy(self.o.tokens))
        out["ln"].copy_(torch.from_numpy(self.o.accept_len))
        out["st"].copy_(torch.from_numpy(self.o.status))
        self.made += 1
        return 0


def test_fewer_steps_than_input_sets():
    ci = synth.tiny_exact_v32()
    o = oracle.greedy(ci.target, ci.tokens, ci.dtype)
    for steps, sets in ((3, 8), (8, 8), (20, 8), (1, 5)):
        lib = Calls(o)
        case = lib.case = bench.Case(lib, "greedy", ci, sets, torch, "cpu")
        for out in case.outputs:  # what memory held before
            for t in out.values():
                t.fill_(99)
        case.run(steps, stream=0)
        r = bench.check_outputs("greedy", case.snapshot(steps), o)
        assert r["mismatched_requests"] == 0 and r["calls_checked"] == min(steps, sets)
        assert abs(r["mean_accept_len"] - o.accept_len.mean()) < 1e-12
