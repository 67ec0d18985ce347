// Shared by the files of the C ABI (defined in ep_api.cpp): the thread's last error, and the check that a
// stream belongs to the calling thread's current device, which is a gfx950 (and its number of compute units).
#pragma once

namespace ep {

int api_fail(int status, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
void api_clear();
int api_stream(void* stream, int* cus = nullptr);

}  // namespace ep
