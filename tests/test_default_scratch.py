"""Default scratch of the W8A8 and mixture-of-experts bindings between host
threads (no GPU: the streams' handles are stood in for)."""
import threading

import torch

from group_wise_affine_quant_b200 import api


def test_host_threads_on_one_stream_have_scratch_of_their_own(monkeypatch):
    """Two threads take scratch at the same time for one stream, then one needs
    more: what the other holds stays its own."""
    monkeypatch.setattr(api, "_stream_of", lambda dev: 7)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    x = torch.zeros((1, 16))
    meet = threading.Barrier(2)
    got = [None, None]

    def run(j):
        got[j] = [api._workspace(None, x, 4096, True)]
        meet.wait()
        if j == 1:
            got[j].append(api._workspace(None, x, 3 << 20, True))
        meet.wait()
        if j == 0:
            got[j].append(api._workspace(None, x, 4096, True))

    threads = [threading.Thread(target=run, args=(j,)) for j in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()

    def span(entry):
        address, size = entry[-2:]
        return address, address + size
    for a in got[0]:
        for b in got[1]:
            (a0, a1), (b0, b1) = span(a), span(b)
            assert a1 <= b0 or b1 <= a0
    assert span(got[0][0]) == span(got[0][1])           # a thread's own buffer is kept
    assert span(got[1][1])[1] - span(got[1][1])[0] >= 3 << 20


def test_scratch_stays_alive_until_the_launch(monkeypatch):
    """What a call is given includes the buffer, so that a larger call in between
    does not hand its memory back."""
    monkeypatch.setattr(api, "_stream_of", lambda dev: 8)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    x = torch.zeros((1, 16))
    buf, address, size = api._workspace(None, x, 4096, True)
    api._workspace(None, x, 3 << 20, True)
    assert buf.data_ptr() == address and buf.numel() == size
    assert int(buf.count_nonzero()) == 0
    space = api.Workspace()
    buf, address, size = api._workspace(space, x, 4096, True)
    space.get(x.device, 3 << 20)
    assert buf.data_ptr() == address and buf.numel() == size
