"""Workspaces of a given room, and streams bound to them."""
import torch


def workspace(room):
    """A workspace to bind to a stream in which a call finds `room` bytes: 256 before them are not for its use, nor are
    4096 more where it has as many."""
    return torch.zeros(256 + room + (4096 if room >= 4096 else 0), dtype=torch.uint8, device="cuda")


class Bound:
    """A stream with a workspace of its own, current inside."""

    def __init__(self, dg, room):
        self.dg, self.ws, self.stream = dg, workspace(room), torch.cuda.Stream()

    def __enter__(self):
        torch.cuda.synchronize()
        self.dg.dg_bind_stream_workspace(self.stream, self.ws)
        self.context = torch.cuda.stream(self.stream)
        self.context.__enter__()
        return self.stream

    def __exit__(self, *error):
        torch.cuda.synchronize()
        self.context.__exit__(*error)
        self.dg.dg_bind_stream_workspace(self.stream, None)
