/* The message msim_last_error(NULL) returns, set by the calls that have no
 * context.  Neither function throws; without memory the message is empty. */
#ifndef MSIM_ERROR_H
#define MSIM_ERROR_H

__attribute__((visibility("hidden"))) void msim_set_error(const char *what) noexcept;
__attribute__((visibility("hidden"))) void msim_set_error2(const char *what, const char *why) noexcept;

#endif
