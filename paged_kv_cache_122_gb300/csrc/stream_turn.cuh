// A stream's turn on the host: calls of several kernels that share scratch.
#pragma once

#include <cstdint>

namespace pk {

// While one lives, no other thread has one for the same device and stream.  The kernels
// of an attention call hand partial results on in a workspace; calls that share it are
// ordered on one stream, but two host threads could queue the first kernels of both
// before the second kernels.  A turn keeps a call's kernels next to each other.  (By
// stream, not by workspace: who waits would wait for the stream's queue anyway, so that a
// launch that blocks holds up nobody on another stream.)  Allocates nothing.
class StreamTurn {
  public:
    StreamTurn(int device, const void *stream);
    ~StreamTurn();
    StreamTurn(const StreamTurn &) = delete;
    StreamTurn &operator=(const StreamTurn &) = delete;

  private:
    int device_;
    uintptr_t stream_;
    StreamTurn *next_;      // of all turns that are being taken
};

}  // namespace pk
