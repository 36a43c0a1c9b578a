"""Host logic of the head operators' torch calls, without a GPU."""
import pytest

import draft_verification_row_amd as sv
from draft_verification_row_amd import heads


@pytest.mark.parametrize("wrap", [1 << 32, 3 << 32, 1 << 31])
def test_sizes_past_32_bits_are_refused(wrap):
    """Sizes that a 32-bit argument would take for small ones."""
    for query, sizes in (("spec_logprobs_workspace_bytes", [1, 6, 100, 5]),
                         ("spec_draft_kl_workspace_bytes", [1, 2, 3, 100]),
                         ("spec_linear_workspace_bytes", [1, 4, 8, 16]),
                         ("spec_linear_grad_workspace_bytes", [1, 4, 8, 16])):
        assert heads._workspace_bytes(query, *sizes) > 0
        for i in (1, 2, 3):
            with pytest.raises(sv.SpecVerifyError):
                heads._workspace_bytes(query, *(n + wrap * (j == i) for j, n in enumerate(sizes)))
                print("not refused:", query, i)


def test_a_capture_on_another_device_is_seen(monkeypatch):
    """Tensors of device 1 while device 0 is current: device 1's stream
    decides whether a call is captured and gets a workspace of its own."""
    import torch
    state = {"device": 0, "capturing": {1}}

    class device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, state["device"] = state["device"], self.index

        def __exit__(self, *_):
            state["device"] = self.before

    monkeypatch.setattr(torch.cuda, "current_device", lambda: state["device"])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["device"] in state["capturing"])
    monkeypatch.setattr(heads, "_stream", lambda index: 7)
    made = []
    monkeypatch.setattr(torch, "zeros", lambda n, **k: made.append(k["device"]) or torch.empty(n, dtype=torch.uint8))
    monkeypatch.setattr(heads, "_workspaces", {})
    one, two = (heads._zeroed(torch.device("cuda", 1), 256) for _ in range(2))
    assert one is not two and len(made) == 2 and not heads._workspaces and state["device"] == 0
    three, four = (heads._zeroed(torch.device("cuda", 0), 256) for _ in range(2))  # not captured: kept
    assert three is four and list(heads._workspaces) == [(0, 7)]


@pytest.mark.parametrize("taken", ["as is", "cast", "viewed", "looked up", "cast, looked up and viewed"])
def test_a_capture_refuses_leaves_behind_one_input_operators(monkeypatch, taken):
    """A weight kept in float32 and cast for each call, a view of it, an
    embedding's rows: the leaf behind is the one whose node counts."""
    import torch
    now = {"stream": 1, "capturing": False}
    monkeypatch.setattr(heads, "_stream", lambda index: now["stream"])
    monkeypatch.setattr(heads, "_capturing", lambda index: now["capturing"])
    leaf = torch.ones(6, 4, requires_grad=True)
    take = {"as is": lambda t: t, "cast": lambda t: t.to(torch.float64), "viewed": lambda t: t.t().reshape(4, 6).t(),
            "looked up": lambda t: t[torch.tensor([1, 5])],
            "cast, looked up and viewed": lambda t: t.double()[torch.tensor([1, 5])].contiguous().view(2, 4)}[taken]

    def call():  # an operator of two inputs, one of them new
        out = take(leaf) * torch.ones(4, requires_grad=True)
        heads._mark_leaves(out)
        return out

    kept = call()
    now.update(stream=2)
    call()                                  # eager: any stream
    now.update(capturing=True)
    with pytest.raises(sv.SpecVerifyError):
        call()
    now.update(stream=1)
    call()                                  # captured on the same stream
    del kept
    now.update(stream=2)
    call()                                  # the graphs are gone
