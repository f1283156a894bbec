// device_status.h -- what the kernels' status words say to the caller.
//
// Each kernel that can give up or meet bad data has a word of its own: 0, or
// one of the codes below.  One call reports all of them, so the gravest has
// to win, and none may pass for success.  (No CUDA here: plain C++.)
#pragma once

namespace wildcat {

// A word's code for the caller: 0, an expired wait (5), a slot, page id, length
// or ring state out of range (1); any other word means that a kernel could not run
// as built and left its output unwritten (3).
constexpr int device_status_code(int word) { return word == 0 || word == 5 || word == 1 ? word : 3; }

// The graver of two codes: an expired wait, then a kernel that did not run (both leave
// outputs incomplete), then bad data (such accesses were skipped).
constexpr int graver_device_status(int a, int b) {
    const int order[] = {5, 3, 1};
    for (const int code : order)
        if (a == code || b == code) return code;
    return 0;
}

}  // namespace wildcat
