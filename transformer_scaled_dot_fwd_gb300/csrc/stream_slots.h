// Which work counter a stream's launches use (host).
#pragma once

namespace attn {

// N slots handed to streams by their ids, which are never used twice.  A stream keeps
// its slot, so launches that share one follow each other in their stream; the slot of
// the stream that has launched nothing for the longest time goes to a new stream when
// all are taken.  The caller holds a lock.
template <int N>
class StreamSlots {
  public:
    int of(unsigned long long stream) {
        ++turn_;
        if (last_ < n_ && id_[last_] == stream) {
            used_[last_] = turn_;
            return last_;
        }
        int oldest = 0, at = 0;
        while (at < n_ && id_[at] != stream) {
            if (used_[at] < used_[oldest]) oldest = at;
            ++at;
        }
        if (at == n_) {
            if (n_ < N)
                ++n_;
            else
                at = oldest;
            id_[at] = stream;
        }
        used_[at] = turn_;
        return last_ = at;
    }

  private:
    unsigned long long id_[N] = {}, used_[N] = {}, turn_ = 0;
    int n_ = 0, last_ = 0;
};

}  // namespace attn
