"""Device memory that calls lend each other."""

from __future__ import annotations

import torch

# The current stream's handle by device index, the current device and whether
# its stream is being captured, without building objects or looking at whether
# the GPU is initialised (1.1 us a call against 1.4).
_raw_stream = torch._C._cuda_getCurrentRawStream
_device_index = torch._C._cuda_getDevice
_stream_capturing = torch._C._cuda_isCurrentStreamCapturing


def _capturing(device: torch.device) -> bool:
    """Whether the device's current stream is being captured into a graph."""
    if device.index == _device_index():
        return _stream_capturing()
    with torch.cuda.device(device):
        return _stream_capturing()


class GrowingBlock:
    """One block of device memory, grown to the largest request and never
    shrunk.  Kernels use it in stream order, so it serves one stream at a time.

    * What is captured into a graph gets memory of its own, from the graph's
      pool: a replay uses the addresses of the capture, and by then this block
      may have been replaced by a larger one and its memory be another tensor's.
    * A block used on another stream than it was allocated on goes back to the
      allocator only behind that stream's work.
    """

    def __init__(self):
        self._block: torch.Tensor | None = None
        self._stream = 0  # that the block was allocated on

    @property
    def nbytes(self) -> int:
        return 0 if self._block is None else self._block.numel()

    def take(self, nbytes: int, device) -> torch.Tensor:
        """At least ``nbytes`` bytes (one at the least), as uint8."""
        dev = device if isinstance(device, torch.device) else torch.device(device)
        stream = 0
        if dev.type == "cuda":
            if dev.index is None:
                dev = torch.device("cuda", torch.cuda.current_device())
            if _capturing(dev):
                return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
            stream = _raw_stream(dev.index)
        block = self._block
        if block is None or block.numel() < nbytes or block.device != dev:
            self._block = block = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
            self._stream = stream
        elif stream != self._stream:
            block.record_stream(torch.cuda.current_stream(dev))
        return block
